// rope_stream.cuh -- the rotation of many rows, through shared memory: rows come and go by
// bulk copies, so that the bytes in flight take no registers.  Every warp has a ring of
// stages of its own, so that no warp waits for another; a stage holds the rows of q, k and
// v and the angles of a few tokens, each brought in, and taken out, by the lane that the
// token belongs to; the warp turns them in place; rows of V only pass through.
#pragma once

#include "rope.cuh"
#include "sm100_ptx.cuh"

namespace attn {

constexpr int kStreamWarps = 8;  // the most of a block
constexpr int kStreamMost = 4;   // stages of a warp, at most

struct StreamShape {
    int warps, stages, tokens;  // of a block, of a warp, of a stage
    int q, k, v, trig;          // bytes of a token's rows, and of its cosines
    int k_at, v_at, c_at, row;  // where they are in its part of a stage, and its size
    int items, lanes;           // of a head; threads along it
    long long rows;             // of the buffers
};

// What a stage's tokens are: written by their lanes, read by all threads.
struct StreamToken {
    int pos;    // -1: outside the table
    int kind;   // 0 none, 1 a row, 2 a padded one
};

template <typename T, int VEC, bool ADJ, bool PAGED>
__device__ __forceinline__ void rope_stream(const RopeArgs &a, const StreamShape &g, uint8_t *smem,
                                            StreamToken (*token)[kStreamMost][32],
                                            uint64_t (*full)[kStreamMost], uint32_t block, uint32_t blocks) {
    using namespace sm100;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *ring = smem + (size_t)warp * g.stages * g.tokens * g.row;
    if (warp >= g.warps) return;
    const uint32_t sbase = smem_addr(ring);
    auto bar = [&](int s) { return smem_addr(full[warp] + s); };
    if (lane < g.stages) {
        mbar_init(bar(lane), 32);
        fence_mbar_init();
    }
    __syncwarp();
    const long long step = (long long)blocks * g.warps * g.tokens;
    const long long first = ((long long)block * g.warps + warp) * g.tokens;
    const int count = first < g.rows ? (int)((g.rows - first + step - 1) / step) : 0;  // stages of work
    T *qo = static_cast<T *>(a.qo), *ko = static_cast<T *>(a.ko), *vo = static_cast<T *>(a.vo);

    // lane l brings in and takes out token l of each stage
    int issued = 0;         // loads
    int b = 0, b_end = -1;  // packed rows: the sequence found last, and its end
    long long krows[kStreamMost];  // rows of the pools of the stages' tokens (registers: see below)
    auto load = [&](int n) {
        issued = n + 1;
        const int s = n % g.stages;
        const uint32_t at = sbase + (uint32_t)((s * g.tokens + lane) * g.row);
        const long long row = first + n * step + lane;
        StreamToken t = {-1, 0};
        uint32_t bytes = 0;
        RopeSeq sq = {};
        int i = 0, bb = 0;
        if (lane < g.tokens && row < g.rows) {
            if (a.cu != nullptr) {  // rows ascend: so do sequences
                if (row >= b_end) {  // the first sequence that ends behind it
                    int lo = b, hi = a.B;
                    while (lo < hi) {
                        const int mid = (lo + hi) >> 1;
                        if (row >= __ldg(a.cu + mid + 1)) lo = mid + 1;
                        else hi = mid;
                    }
                    b = lo;
                    b_end = b < a.B ? __ldg(a.cu + b + 1) : 0;
                }
                bb = b;
                if (b < a.B) {
                    sq = rope_seq(a, b);
                    const long long d = row - sq.row0;
                    if (d >= 0 && d < sq.n) t.kind = 1;
                    i = (int)d;
                }
            } else {
                bb = (int)(row / a.N);
                i = (int)(row - (long long)bb * a.N);
                sq = rope_seq(a, bb);
                t.kind = i < sq.n ? 1 : 2;
            }
        }
        long long krow = row;
        if (t.kind == 1) {
            t.pos = rope_position(a, sq, i);
            if (PAGED) krow = rope_cache_row(a, bb, (long long)sq.len + i);
            bytes = g.q + g.k + (krow >= 0 ? g.v : 0) + (t.pos >= 0 ? 2 * g.trig : 0);
        }
        token[warp][s][lane] = t;
        mbar_arrive_expect_tx(bar(s), bytes);
        if (t.kind == 1) {
            if (g.q) bulk_load(at, static_cast<const T *>(a.q) + row * a.q_stride, g.q, bar(s));
            if (g.k) bulk_load(at + g.k_at, static_cast<const T *>(a.k) + row * a.k_stride, g.k, bar(s));
            if (g.v && krow >= 0) bulk_load(at + g.v_at, static_cast<const T *>(a.v) + row * a.v_stride, g.v, bar(s));
            if (g.trig && t.pos >= 0) {
                const long long p = (long long)t.pos * (a.rot >> 1);
                bulk_load(at + g.c_at, a.cos + p, g.trig, bar(s));
                bulk_load(at + g.c_at + g.trig, a.sin + p, g.trig, bar(s));
            }
        }
#pragma unroll
        for (int k = 0; k < kStreamMost; ++k)
            if (k == s) krows[k] = krow;
    };
    for (int n = 0; n < g.stages && n < count; ++n) load(n);
    const int heads = (g.q ? a.Hq : 0) + (g.k ? a.Hkv : 0);  // side by side in a stage
    const int hstep = 32 / g.lanes, h0 = lane / g.lanes, c0 = lane - h0 * g.lanes;
    bool ok = true;
    for (int n = 0; n < count; ++n) {
        const int s = n % g.stages;
        // (a wait that runs out: nothing more is computed, and the copies are waited for)
        ok = __all_sync(0xffffffffu, mbar_wait_within(bar(s), (uint32_t)(n / g.stages) & 1u, a.wait_ns));
        if (!ok) break;
        uint8_t *part = ring + (size_t)s * g.tokens * g.row;
        for (int k = 0; k < g.tokens; ++k) {
            const StreamToken t = token[warp][s][k];
            uint8_t *mine = part + k * g.row;
            if (t.kind == 0) continue;
            if (t.kind == 2) {  // zeros; a row of q is whole vectors of 16 bytes
                for (int e = lane * 16; e < g.q; e += 512)
                    *reinterpret_cast<uint4 *>(mine + e) = make_uint4(0, 0, 0, 0);
                continue;
            }
            if (h0 >= hstep) continue;
            for (int c = c0; c < g.items; c += g.lanes) {
                const RopeItem<VEC> it = rope_item<VEC, ADJ>(c, a.rot);
                if (it.trig < 0) break;  // plain columns are where they belong
                Trig<VEC> tr;
                const float *cs = reinterpret_cast<const float *>(mine + g.c_at) + it.trig;
                if (t.pos >= 0) tr.load_from(cs, cs + (a.rot >> 1), a.sign);
                else tr.set_nan();
                T *head = reinterpret_cast<T *>(mine) + h0 * a.D;
#pragma unroll 2
                for (int h = h0; h < heads; h += hstep, head += hstep * a.D) {
                    RowVec<T, VEC> u, w;
                    u.load(head + it.a);
                    w.load(head + it.b);
                    float y[2 * VEC];
                    turn_item<T, VEC, ADJ>(it, u, w, tr, y);
                    u.set(y);
                    w.set(y + VEC);
                    u.store(head + it.a);
                    w.store(head + it.b);
                }
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        {
            const StreamToken t = token[warp][s][lane];
            const uint32_t at = sbase + (uint32_t)((s * g.tokens + lane) * g.row);
            const long long row = first + n * step + lane;
            long long krow = -1;
#pragma unroll
            for (int k = 0; k < kStreamMost; ++k)
                if (k == s) krow = krows[k];
            if (t.kind != 0 && g.q) bulk_store(qo + row * a.Hq * a.D, at, g.q);
            if (t.kind == 1 && krow >= 0) {
                if (g.k) bulk_store(ko + krow * a.Hkv * a.D, at + g.k_at, g.k);
                if (g.v) bulk_store(vo + krow * a.Hkv * a.Dv, at + g.v_at, g.v);
            }
            bulk_commit();
        }
        // the stage before this one: its rows have left by now, or nearly
        if (n > 0 && n - 1 + g.stages < count) {
            bulk_wait_read<1>();
            __syncwarp();
            load(n - 1 + g.stages);
        }
    }
    // what is on its way in has landed, and what is on its way out is written
    if (!ok) {
        if (lane == 0) report_status(a.status, kStatusTimeoutRope);
        for (int n = max(0, issued - g.stages); n < issued; ++n)
            mbar_wait_drain(bar(n % g.stages), (uint32_t)(n / g.stages) & 1u);
    }
    bulk_wait0();
}

// Stages of `blocks` blocks of up to `warps` warps with `bytes` each; false: rows too long.
template <typename T, int VEC>
bool stream_shape(const RopeArgs &a, long long bytes, int warps, int blocks, StreamShape &g) {
    const long long es = sizeof(T);
    const long long q = a.qo ? a.Hq * (long long)a.D * es : 0, k = a.ko ? a.Hkv * (long long)a.D * es : 0;
    const long long v = a.vo ? a.Hkv * (long long)a.Dv * es : 0, trig = a.rot / 2 * 4LL;
    const long long row = q + k + v + 2 * trig;
    if (row == 0 || row * 4 > bytes) return false;  // two warps of two stages
    g.q = (int)q;
    g.k = (int)k;
    g.v = (int)v;
    g.trig = (int)trig;
    g.k_at = g.q;
    g.v_at = g.q + g.k;
    g.c_at = g.v_at + g.v;
    g.row = (int)row;
    // as many warps as two stages of a token leave room for, then tokens, then stages; few
    // rows: stages of fewer tokens, so that no warp's last one is much of its work
    g.warps = (int)(bytes / (2 * row));
    if (g.warps > warps) g.warps = warps;
    g.rows = a.cu ? a.total : (long long)a.B * a.N;
    const long long ring = bytes / g.warps, mine = (g.rows - 1) / (blocks * (long long)g.warps) + 1;
    long long tokens = ring / (2 * row);
    if (tokens > 32) tokens = 32;
    long long rounds = (mine + tokens - 1) / tokens;
    if (rounds < 4) rounds = 4;
    g.tokens = (int)((mine + rounds - 1) / rounds);
    const long long stages = ring / (row * g.tokens);
    g.stages = (int)(stages < kStreamMost ? stages : kStreamMost);
    g.items = rope_items<VEC>(a.D, a.rot);
    g.lanes = g.items < 32 ? g.items : 32;
    return true;
}

}  // namespace attn
