// checks.hpp -- host-side argument checks of the block operators' entry points:
// sizes, pointers, overlaps, workspaces and the vector width a layout allows.
// (The scans' entry points have theirs in api.hip.)
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "miscan.h"

namespace miscan {

inline size_t elem_size(mi_dtype dt) { return dt == MI_F32 ? 4 : 2; }
inline bool dtype_known(mi_dtype dt) { return dt == MI_F32 || dt == MI_BF16 || dt == MI_F16; }

// a*b*c*d into *out without int64 overflow; all factors non-negative.
inline bool mul_ok(int64_t a, int64_t b, int64_t c, int64_t d, int64_t *out) {
    int64_t r;
    if (__builtin_mul_overflow(a, b, &r)) return false;
    if (__builtin_mul_overflow(r, c, &r)) return false;
    if (__builtin_mul_overflow(r, d, &r)) return false;
    *out = r;
    return true;
}

// Whether one launch can hold `groups` workgroups: a grid counts its threads in 32 bits.
inline bool launch_fits(int64_t groups, int64_t threads) { return groups <= (int64_t)0xffffffffll / threads; }

struct Buf {
    const void *p;
    int64_t bytes;
};

inline bool overlaps(const Buf &x, const Buf &y) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(x.p), b0 = reinterpret_cast<uintptr_t>(y.p);
    return a0 < b0 + (uintptr_t)y.bytes && b0 < a0 + (uintptr_t)x.bytes;
}

inline mi_status check_ws(void *ws, size_t ws_bytes, size_t need, const Buf *bufs, int n) {
    if (ws == nullptr || ws_bytes < need) return MI_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(ws) % 256 != 0) return MI_ERR_INVALID_ARG;
    Buf w{ws, (int64_t)ws_bytes};
    for (int i = 0; i < n; ++i)
        if (overlaps(w, bufs[i])) return MI_ERR_INVALID_ARG;
    return MI_OK;
}

// The buffers of a call, inputs and outputs apart, with each one's alignment.
// need() takes a buffer the call cannot do without, opt() one that may be NULL.
// Empty buffers are skipped.
struct BufList {
    static constexpr int MAX = 24;
    Buf b[MAX];
    int n = 0;
    bool bad = false;  // a missing or misaligned buffer
    BufList &need(const void *p, int64_t bytes, size_t align) {
        if (bytes <= 0) return *this;
        if (p == nullptr || reinterpret_cast<uintptr_t>(p) % align != 0 || n == MAX) bad = true;
        else b[n++] = Buf{p, bytes};
        return *this;
    }
    BufList &opt(const void *p, int64_t bytes, size_t align) { return p == nullptr ? *this : need(p, bytes, align); }
};

// Missing, misaligned or overlapping buffers: an output overlaps nothing else.
inline mi_status check_lists(const BufList &in, const BufList &out) {
    if (in.bad || out.bad) return MI_ERR_INVALID_ARG;
    for (int i = 0; i < out.n; ++i) {
        for (int j = 0; j < in.n; ++j)
            if (overlaps(out.b[i], in.b[j])) return MI_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlaps(out.b[i], out.b[j])) return MI_ERR_INVALID_ARG;
    }
    return MI_OK;
}

inline mi_status check_ws_lists(void *ws, size_t ws_bytes, size_t need, const BufList &in, const BufList &out) {
    const mi_status st = check_ws(ws, ws_bytes, need, in.b, in.n);
    return st != MI_OK ? st : check_ws(ws, ws_bytes, need, out.b, out.n);
}

// Widest vector (elements per lane) such that D is a multiple of it and every
// pointer is aligned to the access width; 16-byte accesses at most.
inline int pick_vec(int64_t D, size_t esize, const Buf *bufs, int n) {
    const int maxv = (int)(16 / esize);
    for (int v = maxv; v > 1; v /= 2) {
        if (D % v != 0) continue;
        bool ok = true;
        for (int i = 0; i < n && ok; ++i)
            ok = reinterpret_cast<uintptr_t>(bufs[i].p) % (v * esize) == 0;
        if (ok) return v;
    }
    return 1;
}

}  // namespace miscan
