// kernel_decode.cu -- split-KV tensor-core decode for bf16 / fp16: its launches, and the
// choice of its splits (the kernel: decode.cuh).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstring>
#include <type_traits>

#include "decode.cuh"
#include "launch.h"

namespace attn {
namespace {

template <typename T, int D, int DV, int NT>
int launch_decode_t(const AttnParams &p, cudaStream_t stream) {
    constexpr int smem = kStages * kTK * (D + DV) * 2 + 64;  // ring + TMA barriers
    // K / V by TMA as flat [rows][Hkv][D] arrays (rows: B * K padded, Tk
    // packed, the page pool when paged); cp.async where pages hold fewer
    // than 64 rows or a tensor map cannot be made
    const bool bf16 = std::is_same<T, __nv_bfloat16>::value;
    const long long rows = p.block_table ? (long long)p.num_pages * p.page_size
                                         : (p.cu_q ? p.Tk : (long long)p.B * p.K);
    CUtensorMap tk, tv;
    memset(&tk, 0, sizeof(tk));
    memset(&tv, 0, sizeof(tv));
    bool tma = (!p.block_table || p.page_size >= kTK) && rows > 0 && rows < (1LL << 31);
    if (tma) {
        tma = make_tma_map_4d(&tk, p.k, bf16, (uint64_t)D, p.Hkv, (uint64_t)rows, 1, 1, kTK) == 0 &&
              make_tma_map_4d(&tv, p.v, bf16, (uint64_t)DV, p.Hkv, (uint64_t)rows, 1, 1, kTK) == 0;
        if (!tma) clear_error();
    }
    auto kern = tma ? decode_kernel<T, D, DV, NT, kLoadTma, false>
                    : (p.block_table ? decode_kernel<T, D, DV, NT, kLoadAsyncPaged, false>
                                     : decode_kernel<T, D, DV, NT, kLoadAsync, false>);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) {
        set_error("decode kernel: cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        return 3;
    }
    dim3 grid((unsigned)p.nsplit, (unsigned)(p.B * p.Hkv));
    kern<<<grid, kDecodeThreads, smem, stream>>>({p}, tk, tv);
    e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("decode kernel launch: %s", cudaGetErrorString(e));
        return 3;
    }
    count_launch();
    return 0;
}

template <typename T, int D, int DV>
int launch_decode_nt(const AttnParams &p, cudaStream_t stream) {
    return p.Q * p.G <= 8 ? launch_decode_t<T, D, DV, 1>(p, stream)
                          : launch_decode_t<T, D, DV, 2>(p, stream);
}

template <typename T>
int launch_decode_dims(const AttnParams &p, cudaStream_t stream) {
    if (p.D == 128 && p.Dv == 128) return launch_decode_nt<T, 128, 128>(p, stream);
    if (p.D == 256 && p.Dv == 256) return launch_decode_nt<T, 256, 256>(p, stream);
    if (p.D == 64 && p.Dv == 64) return launch_decode_nt<T, 64, 64>(p, stream);
    if (p.D == 128 && p.Dv == 64) return launch_decode_nt<T, 128, 64>(p, stream);
    return launch_decode_nt<T, 64, 128>(p, stream);
}

}  // namespace

bool decode_supported(const AttnParams &p, int dtype) {
    if (dtype != 1 && dtype != 2) return false;
    // head dims 64 / 128 in any pair, or 256 / 256 (one block an SM: 192 KB of ring)
    const bool small = (p.D == 64 || p.D == 128) && (p.Dv == 64 || p.Dv == 128);
    if (!small && !(p.D == 256 && p.Dv == 256)) return false;
    if ((long long)p.Q * p.G > 16 || p.Q < 1) return false;
    return (long long)p.B * p.Hkv <= 65535;
}

int decode_split_len(const AttnParams &p, int nsm) {
    // Small splits balance sequences of very different lengths; fewer, longer
    // splits when the (sequence, KV head) units already fill the SMs.
    if (nsm < 1) nsm = 1;  // a failed device query must not divide by zero
    const long long units = (long long)p.B * p.Hkv;
    long long len = ((long long)p.K * units + 4LL * nsm - 1) / (4LL * nsm);
    len = (len + kTK - 1) / kTK * kTK;
    if (len < 128) len = 128;
    if (len > 1024) len = 1024;
    return (int)len;
}

int launch_decode(const AttnParams &p, int dtype, cudaStream_t stream) {
    if (p.nsplit > 0x7fffffff / 2) {
        set_error("decode kernel: too many splits");
        return 2;
    }
    if (dtype == 2) return launch_decode_dims<__nv_bfloat16>(p, stream);
    return launch_decode_dims<__half>(p, stream);
}

}  // namespace attn
