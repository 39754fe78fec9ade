// What the operators' C entry points share: the device, its status word,
// argument checks.
#pragma once

#include "det_gemm.h"

#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>
#include <initializer_list>

namespace deto {

constexpr int64_t kMaxRows = (int64_t{1} << 31) - 4096;

struct Device {
    bool init = false;
    det_gemm_status status = DET_GEMM_OK;
    int sms = 0;
    int *word = nullptr;             // the status word that kernels set
};

// The current device, or why it cannot be used.
det_gemm_status device(Device **out);
// Keeps the error's text for det_gemm_last_error_detail and returns st.
det_gemm_status fail(det_gemm_status st, cudaError_t e, const char *where);
// Known once device() has succeeded.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();
unsigned long long timeout_ns();     // bound of a kernel's waits
bool timeout_forced();               // the test hook is on

// A strided array: `rows` rows of `cols` elements, pitch `ld`, element size
// `es`, in `mats` matrices `gap` elements apart. `align`: the base's and the
// pitch's alignment in bytes.
struct Arr {
    const void *p;
    int64_t rows, cols, ld;
    int es, align;
    int64_t mats = 1, gap = 0;
    int64_t bytes() const { return ((mats - 1) * gap + (rows - 1) * ld + cols) * es; }
    bool empty() const { return rows <= 0 || cols <= 0 || mats <= 0; }
};

// More bytes than there are addresses; what is below fits 64-bit arithmetic.
constexpr double kMaxBytes = 1ull << 57;

inline det_gemm_status check(const Arr &a)
{
    if (a.empty()) return DET_GEMM_OK;
    if (!a.p || a.ld < a.cols || a.ld > (int64_t{1} << 36)) return DET_GEMM_ERR_INVALID_ARG;
    if ((static_cast<double>(a.mats - 1) * a.gap + static_cast<double>(a.rows - 1) * a.ld + a.cols) * a.es > kMaxBytes)
        return DET_GEMM_ERR_INVALID_ARG;
    if (a.mats > 1 && (a.gap < (a.rows - 1) * a.ld + a.cols || a.gap > (int64_t{1} << 40))) return DET_GEMM_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(a.p) % a.align != 0 || a.ld * a.es % a.align != 0) return DET_GEMM_ERR_ALIGNMENT;
    if (a.mats > 1 && a.gap * a.es % a.align != 0) return DET_GEMM_ERR_ALIGNMENT;
    return DET_GEMM_OK;
}

inline bool overlap(const Arr &a, const Arr &b)
{
    if (a.empty() || b.empty() || !a.p || !b.p) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + static_cast<uintptr_t>(b.bytes()) && y < x + static_cast<uintptr_t>(a.bytes());
}

// All arrays well formed, and no output overlapping an input or another output.
inline det_gemm_status check_all(std::initializer_list<Arr> in, std::initializer_list<Arr> out)
{
    for (const Arr &a : in) {
        const det_gemm_status s = check(a);
        if (s != DET_GEMM_OK) return s;
    }
    for (const Arr *o = out.begin(); o != out.end(); ++o) {
        const det_gemm_status s = check(*o);
        if (s != DET_GEMM_OK) return s;
        for (const Arr &a : in)
            if (overlap(*o, a)) return DET_GEMM_ERR_INVALID_ARG;
        for (const Arr *b = out.begin(); b != o; ++b)
            if (overlap(*o, *b)) return DET_GEMM_ERR_INVALID_ARG;
    }
    return DET_GEMM_OK;
}

inline Arr bf16(const void *p, int64_t r, int64_t c, int64_t ld) { return Arr{p, r, c, ld, 2, 16}; }
inline Arr vec4(const void *p, int64_t n) { return Arr{p, 1, n, n, 4, 4}; }
inline Arr mat8(const void *p, int64_t r, int64_t c, int64_t ld, int64_t mats = 1, int64_t gap = 0)
{
    return Arr{p, r, c, ld, 1, 16, mats, gap};
}

inline bool ok_size(int64_t v) { return v >= 0 && v <= kMaxRows; }
inline bool launchable(int64_t blocks) { return blocks <= (int64_t{1} << 31) - 1; }
inline cudaStream_t cs(det_gemm_stream s) { return reinterpret_cast<cudaStream_t>(s); }
inline int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace deto
