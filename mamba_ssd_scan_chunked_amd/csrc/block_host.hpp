// Host-side argument checks shared by the operators around the scan.  Internal to the library.
#pragma once
#include "ssd_host.hpp"

namespace ssd_host {

// A tensor argument's span, null or empty ones overlapping nothing.
struct Buf {
    const void* ptr;
    int64_t bytes;
};
// Every output against every input and the outputs after it.
inline int check_alias(const Buf* in, int nin, const Buf* out, int nout) {
    for (int i = 0; i < nout; ++i) {
        for (int j = 0; j < nin; ++j)
            if (overlap(out[i].ptr, out[i].bytes, in[j].ptr, in[j].bytes)) return SSD_ERR_ALIAS;
        for (int j = i + 1; j < nout; ++j)
            if (overlap(out[i].ptr, out[i].bytes, out[j].ptr, out[j].bytes)) return SSD_ERR_ALIAS;
    }
    return SSD_OK;
}

// Sequences of the operators around the scan (P: their problem structs).
template <typename P> inline int check_sequences(const P* p, const int32_t* seq_idx) {
    if (!seq_idx && p->nseqs != p->batch) return SSD_ERR_BAD_SHAPE;
    if (seq_idx && p->batch * p->seqlen > 0 && p->nseqs < 1) return SSD_ERR_BAD_SHAPE;
    return SSD_OK;
}

}  // namespace ssd_host
