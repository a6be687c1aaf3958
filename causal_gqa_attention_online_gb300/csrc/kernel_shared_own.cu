// kernel_shared_own.cu -- the keys that each of a batch's sequences has alone, where few
// query rows attend to them (the kernel: decode.cuh): beside the tcgen05 kernel of the
// shared keys, which it follows as its programmatic dependent, so that its blocks fill the
// SMs as that kernel's shares end.
#include <cuda.h>

#include <cstring>

#include "decode.cuh"
#include "launch.h"

namespace attn {
namespace {

template <typename T, int D, int DV, int NT> int launch_t(const SharedArgs &a, bool bf16, cudaStream_t stream) {
    constexpr int smem = kOwnStages * kTK * (D + DV) * 2 + 64;  // ring + TMA barriers
    const AttnParams &p = a.p;
    const uint64_t rows = (uint64_t)p.num_pages * p.page_size;
    CUtensorMap tk, tv;
    memset(&tk, 0, sizeof(tk));
    memset(&tv, 0, sizeof(tv));
    const bool tma = p.page_size >= kTK;
    if (tma) {
        int rc = make_tma_map_4d(&tk, p.k, bf16, D, p.Hkv, rows, 1, 1, kTK);
        if (rc == 0) rc = make_tma_map_4d(&tv, p.v, bf16, DV, p.Hkv, rows, 1, 1, kTK);
        if (rc) return rc;
    }
    auto kern = tma ? decode_kernel<T, D, DV, NT, kLoadTma, true> : decode_kernel<T, D, DV, NT, kLoadAsyncPaged, true>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) {
        set_error("own-keys kernel: cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        return 3;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.own_splits, (unsigned)(p.B * p.Hkv));
    cfg.blockDim = dim3(kDecodeThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, a, tk, tv);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("own-keys kernel launch: %s", cudaGetErrorString(e));
        return 3;
    }
    count_launch();
    return 0;
}

template <typename T, int D, int DV> int launch_nt(const SharedArgs &a, bool bf16, cudaStream_t stream) {
    return a.p.Q * a.p.G <= 8 ? launch_t<T, D, DV, 1>(a, bf16, stream) : launch_t<T, D, DV, 2>(a, bf16, stream);
}

template <typename T> int launch_dims(const SharedArgs &a, bool bf16, cudaStream_t stream) {
    if (a.p.D == 128 && a.p.Dv == 128) return launch_nt<T, 128, 128>(a, bf16, stream);
    if (a.p.D == 64 && a.p.Dv == 64) return launch_nt<T, 64, 64>(a, bf16, stream);
    if (a.p.D == 128) return launch_nt<T, 128, 64>(a, bf16, stream);
    return launch_nt<T, 64, 128>(a, bf16, stream);
}

}  // namespace

// (decode.cuh has at most 16 rows.  More take tiles of 128 on the tcgen05 kernel, most of them
// empty: 64 sequences over 4096 keys and 500 of their own, 8 heads of 4 rows of 128, take 74 us
// for 4 tokens each and 86 for 5; over 32768, 159 and 240.)
bool own_decode_supported(const AttnParams &p) {
    return (p.D == 64 || p.D == 128) && (p.Dv == 64 || p.Dv == 128) && (long long)p.Q * p.G <= 16 &&
           (long long)p.B * p.Hkv <= 65535 && (uint64_t)p.num_pages * p.page_size < (1ull << 31);
}

int launch_own_decode(const SharedArgs &a, bool bf16, cudaStream_t stream) {
    return bf16 ? launch_dims<__nv_bfloat16>(a, true, stream) : launch_dims<__half>(a, false, stream);
}

}  // namespace attn
