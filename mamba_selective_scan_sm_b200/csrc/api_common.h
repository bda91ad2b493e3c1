// Argument checks shared by the host code of the C ABI.
#pragma once

#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "../../include/ssm.h"
#include "launch.h"

namespace ssm {

inline ssm_status_t api_fail(ssm_status_t s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    set_error_detail(buf);
    return s;
}

inline ssm_status_t api_ok() {
    set_error_detail("");
    return SSM_OK;
}

inline ssm_status_t api_cuda(cudaError_t e, const char* what) {
    return api_fail(SSM_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

inline bool is_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

inline bool ranges_overlap(const void* a, size_t na, const void* b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    auto x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// A pointer argument: its alignment, and the bytes it spans (0 where they are not checked).
// Views in rows: row bytes every step bytes.
struct Arg {
    const void* p;
    size_t align, bytes;
    const char* name;
    size_t row = 0, step = 0;
};

template <int N>
inline ssm_status_t check_aligned(const Arg (&args)[N]) {
    for (const Arg& a : args)
        if (a.p && !is_aligned(a.p, a.align))
            return api_fail(SSM_ERR_MISALIGNED, "%s is not %zu-byte aligned", a.name, a.align);
    return SSM_OK;
}

// Whether two arguments share an element. Two with the same step may interleave (columns of
// one tensor).
inline bool share(const Arg& a, const Arg& b) {
    if (!ranges_overlap(a.p, a.bytes, b.p, b.bytes)) return false;
    const auto pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    const Arg &x = pa >= pb ? a : b, &y = pa >= pb ? b : a;    // x's first row among y's rows
    if (x.step == 0 || x.step != y.step) return true;
    const size_t d = (pa >= pb ? pa - pb : pb - pa) % x.step;
    return d < y.row || x.step - d < x.row;
}

template <int NO, int NI>
inline ssm_status_t check_alias(const Arg (&outs)[NO], const Arg (&ins)[NI]) {
    for (const Arg& o : outs)
        for (const Arg& i : ins)
            if (share(o, i)) return api_fail(SSM_ERR_ALIAS, "%s overlaps %s", o.name, i.name);
    return SSM_OK;
}

template <int N>
inline ssm_status_t check_distinct(const Arg (&outs)[N]) {
    for (int i = 0; i < N; ++i)
        for (int k = 0; k < i; ++k)
            if (share(outs[i], outs[k]))
                return api_fail(SSM_ERR_ALIAS, "%s overlaps %s", outs[i].name, outs[k].name);
    return SSM_OK;
}

inline bool bad_dtype(ssm_dtype_t t) { return t != SSM_F32 && t != SSM_BF16; }
inline int size_of(ssm_dtype_t t) { return t == SSM_BF16 ? 2 : 4; }

}  // namespace ssm
