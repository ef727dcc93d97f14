// Checks of arguments shared by the C entry points (api.cu, block_api.cu).
#pragma once

#include <utility>

#include "../../include/slra.h"
#include "common.cuh"

namespace slra {

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

inline bool default_split(int64_t D, const int64_t* s, int64_t out[3]) {
    const int64_t c = D / 2;
    if (s[0] == 0 && s[1] == 0 && s[2] == 0) {
        out[1] = c / 3;
        out[2] = c / 3;
        out[0] = c - 2 * (c / 3);
        return true;
    }
    if (s[0] < 0 || s[1] < 0 || s[2] < 0 || s[0] + s[1] + s[2] != c) return false;
    out[0] = s[0]; out[1] = s[1]; out[2] = s[2];
    return true;
}

// Element strides (batch, token, head) of a [B][L][Hh][D] tensor: all zero means contiguous
// (token-major); otherwise positive multiples of `align` elements (16-byte TMA strides), below 2^36.
inline bool strides_of(const int64_t s[3], int64_t L, int64_t Hh, int64_t D, int64_t align, Strides* out) {
    if (s[0] == 0 && s[1] == 0 && s[2] == 0) {
        out->h = D;
        out->l = Hh * D;
        out->b = L * Hh * D;
        return true;
    }
    for (int i = 0; i < 3; ++i)
        if (s[i] <= 0 || s[i] % align != 0 || s[i] >= (int64_t(1) << 36)) return false;
    out->b = s[0];
    out->l = s[1];
    out->h = s[2];
    return true;
}

// Elements from a tensor's first element to one past its last.
inline int64_t extent_elems(const Strides& st, int64_t B, int64_t L, int64_t Hh, int64_t D) {
    return (B - 1) * st.b + (L - 1) * st.l + (Hh - 1) * st.h + D;
}

// True when distinct (batch, token, head) rows of D elements never share an element: taking the
// dimensions by increasing stride, each stride clears everything the smaller ones span.
inline bool rows_disjoint(const Strides& st, int64_t B, int64_t L, int64_t Hh, int64_t D) {
    int64_t s[3] = {st.b, st.l, st.h}, n[3] = {B, L, Hh};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (s[j] < s[i]) { std::swap(s[i], s[j]); std::swap(n[i], n[j]); }
    int64_t span = D;
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) continue;
        if (s[i] < span) return false;
        span += s[i] * (n[i] - 1);
    }
    return true;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// The current device must be an sm_100 part (the kernels are built for sm_100a only).
inline slra_status check_device() {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) { cudaGetLastError(); return SLRA_ERR_NO_DEVICE; }
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
        cudaGetLastError();
        return SLRA_ERR_NO_DEVICE;
    }
    return (major == 10 && minor == 0) ? SLRA_OK : SLRA_ERR_NO_DEVICE;
}

inline slra_status cuda_status(cudaError_t e) { return e == cudaSuccess ? SLRA_OK : SLRA_ERR_CUDA; }

}  // namespace slra
