"""The words that tiles of the gated linear recurrence publish: a word that never came poisons what
is made of it, and no map is lost on its way through a word.  The header's functions as the host
runs them."""
import os
import subprocess

from mamba_ssd_scan_chunked_amd import build

PROGRAM = r"""
#include <cmath>
#include <cstdio>
#include <cstring>
#include "ssd_recurrence_map.hpp"
using namespace ssd;
static int bad = 0;
#define EXPECT(c) do { if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); bad = 1; } } while (0)
static float bits(uint32_t b) { float f; std::memcpy(&f, &b, 4); return f; }
int main() {
    // a word that never came, as a state, as a map alone and between others, packed and not
    EXPECT(std::isnan(state_of(0)));
    const Map lost = map_of(0), one{1.f, 0.f}, half{0.5f, 3.f}, fresh{-1.f, 4.f};
    for (float h : {0.f, 1.f, -2.5f}) {
        EXPECT(std::isnan(apply<false>(lost, h)) && std::isnan(apply<true>(lost, h)));
        EXPECT(std::isnan(apply<false>(then<false>(one, lost), h)));
        EXPECT(std::isnan(apply<true>(then<true>(fresh, lost), h)));
        EXPECT(std::isnan(apply<false>(then<false>(then<false>(half, lost), half), h)));
        // unless a sequence begins behind it
        EXPECT(apply<true>(then<true>(lost, fresh), h) == 4.f);
    }
    // every map's word is there, and gives the map back
    const float values[] = {0.f, -0.f, 1.f, -1.f, 0.25f, 1e-40f, -3e38f, INFINITY, -INFINITY, bits(1)};
    for (float P : values)
        for (float H : values) {
            const uint64_t w = word_of({P, H});
            EXPECT((uint32_t)w != 0);
            const Map m = map_of(w);
            EXPECT(!std::memcmp(&m.P, &P, 4) && !std::memcmp(&m.H, &H, 4));
        }
    for (uint32_t b : {0xffffffffu, 0x7fffffffu, 0x7fc00000u, 0xffc00000u, 0x7f800001u}) {
        const uint64_t w = word_of({bits(b), 2.f});
        EXPECT((uint32_t)w != 0 && std::isnan(map_of(w).P) && map_of(w).H == 2.f);
        EXPECT(std::isnan(map_of(word_of({0.5f, bits(b)})).H));
    }
    for (float h : {0.f, -0.f, 2.f, -1e38f, INFINITY, -INFINITY}) {
        const float s = state_of(word_of({1.f, h}));
        EXPECT(!std::memcmp(&s, &h, 4));
    }
    return bad;
}
"""


def test_words_of_maps(tmp_path):
    src, exe = tmp_path / "map.hip", tmp_path / "map"
    src.write_text(PROGRAM)
    subprocess.run([build.hipcc(), "--offload-host-only", "-O1", "-std=c++17", "-I" + build.CSRC, str(src), "-o", str(exe)],
                   check=True, timeout=300)
    r = subprocess.run([str(exe)], stdout=subprocess.PIPE, text=True, timeout=60, env=dict(os.environ))
    assert r.returncode == 0, r.stdout
