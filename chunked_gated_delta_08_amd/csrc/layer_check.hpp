// layer_check.hpp -- host-side checks shared by the C entries of the layer operators
// (layer_api.cpp, ffn_api.cpp).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdr.h"

namespace layer_check {

inline int status(hipError_t e) { return e == hipSuccess ? GDR_OK : GDR_ERR_LAUNCH; }
inline bool known(int dt) { return dt == GDR_F32 || dt == GDR_F16 || dt == GDR_BF16; }
inline size_t size_of(int dt) { return dt == GDR_F32 ? 4 : 2; }

// A buffer of a call; a null pointer or no bytes overlaps nothing.
struct Buf {
    const void* p;
    size_t bytes, align;
    bool aligned() const { return ((uintptr_t)p & (align - 1)) == 0; }
    bool overlaps(const Buf& o) const {
        if (!p || !o.p || !bytes || !o.bytes) return false;
        const uintptr_t a = (uintptr_t)p, b = (uintptr_t)o.p;
        return a < b + o.bytes && b < a + bytes;
    }
};
// Every buffer aligned to its element; no output on an input or another
// output, but for inputs that it exactly replaces (bit i of `same`: input i).
struct Out {
    Buf b;
    unsigned same;
};
template <int NI, int NO> bool buffers_ok(const Buf (&in)[NI], const Out (&out)[NO]) {
    for (int i = 0; i < NI; i++)
        if (!in[i].aligned()) return false;
    for (int j = 0; j < NO; j++) {
        if (!out[j].b.aligned()) return false;
        for (int i = 0; i < NI; i++) {
            const bool replaces = (out[j].same >> i & 1) && in[i].p == out[j].b.p && in[i].bytes == out[j].b.bytes;
            if (!replaces && out[j].b.overlaps(in[i])) return false;
        }
        for (int k = 0; k < j; k++)
            if (out[j].b.overlaps(out[k].b)) return false;
    }
    return true;
}

inline int check_ws(const void* ws, size_t have, size_t need) {
    if (need == 0) return GDR_OK;
    return !ws || have < need || ((uintptr_t)ws & 15) ? GDR_ERR_WORKSPACE : GDR_OK;
}

}  // namespace layer_check
