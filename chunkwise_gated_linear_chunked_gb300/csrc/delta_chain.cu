// Gated delta rule in chunks of 64 tokens, the chain over a sequence's chunks (see DeltaCell for what the cells hold):
//
//     R = V - e^G K S,   Y = T^ R,   N = beta Y,   o = scale e^G q S + P N,   S <- e^G_end S + (e^(G_end - G) K)^T N
//
// The columns of S do not meet, and 16 of them make one warp's rows: transposed, S' (16 x keys) is the left operand of
// S' K', whose result is the left operand of (T^ R)' = R' T^', whose result is that of S' += N' K.  So the chain of a
// chunk's products stays in the registers of one warp.  A second warp has what is not on the way from one state to the
// next: the output o' = S' q' + N' P' from the first one's rounded S and its Y, and before that the remainders' share of
// S' K'.  Each has 252 of a chunk's 504 products of 16 x 8 x 16 (8 cycles each on a quarter of an SM).
//
// Inputs are exact operands; S, R, N and the cells' matrices go in as a rounded value and its remainder, two products for
// an exact partner and three for another such (the product of two remainders, 2^-18, is left out).
//
// A CTA takes 32 columns where those make fewer CTAs than the GPU has SMs: its four warps have a quarter of the SM each, and
// a chunk takes 1.95 us.  Otherwise 64: shared memory, which every warp's right operands pass, and the quarters are then
// about equally busy, 3.4 us a chunk.  (4 x 2048 tokens of 8 heads, prep included: 87 us with 32 columns, 135 with 64; the
// pack of 16 sequences of 16 heads: 1010 and 934.  Two warps that share 16 columns by keys, and add their partial sums
// through shared memory, were bound by it: 2.7 us a chunk of 32 columns where the products take 1.0.)
//
// Warp matrix instructions and not tcgen05: the chain is bound by its latency, with 32 columns a CTA, and there a
// product's way through tensor memory and shared memory (a commit, a load, a conversion and a store between any two) costs
// more than the products.
#include "delta_chain.cuh"

namespace gla {
namespace {

// SAVE: for the gradients, instead of o its products with dO, the rounded states and rows, Y, and every second state.  The
// gradient of a gate is a sum of o.dO - dv.v over rows that cancel but for what later rows have of earlier ones, so that the
// two have to be of one linear map where they cancel: the diagonals of T^ and T' are exact, P' is P to the bit, and N is an
// operand of three terms where it meets P, and behind the last chunk where it meets K, since the gradient of the final state
// can be of any size (4 x 2048 tokens of 8 heads, a gradient of the final state as large as its values: dg off by 5.8e-6 of
// it; 3.6e-5 with two terms throughout and T^ with its diagonal).
template <typename T, typename To, int KD, int VG, bool SAVE>
__global__ void __launch_bounds__(64 * VG, 1) delta_chain_kernel(const __grid_constant__ ChainMaps maps, DeltaArgs a, int tiles)
{
    typedef ChainShared<KD, VG, SAVE ? 2 : 1, DeltaCell> Shared;
    constexpr int kThreads = 64 * VG;
    constexpr bool kThree = SAVE && std::is_same_v<T, __nv_bfloat16>;   // fp16's second term already ends at the type's last bit
    constexpr size_t kCell = SAVE ? sizeof(DeltaCellBack) : sizeof(DeltaCell);
    extern __shared__ __align__(1024) char raw[];
    Shared &sh = *reinterpret_cast<Shared *>(raw);
    ChainWalk w;
    bars_init(sh.full);
    tc::grid_dep_wait();
    if (!chain_walk(a, tiles, 16 * VG, w))
        return;
    const int tid = threadIdx.x, lane = tid % 32, group = tid / 32 % VG;
    const bool output = tid >= kThreads / 2;
    const int col = w.v0 + 16 * group + lane / 4, two = 2 * (lane % 4);
    const bool on = w.v0 + 16 * group < a.V;   // whole groups of 16 columns
    const size_t state = (w.head * a.K + two) * a.V;

    Power in[2] = {{1.f, 1.f}, {1.f, 1.f}};   // fp16: the powers that the state's columns are held over
    auto chain = [&](typename Shared::Stage &st, float (&s)[KD / 8][4], bool end) {
        const float4 *row = st.cell.row;
        float n[8][4] = {};
        {
            uint32_t s_hi[KD / 16][4];
            if constexpr (kScaled<T>)
                if (lane % 4 == 0) {
                    sh.power[group][lane / 4] = in[0].from;
                    sh.power[group][lane / 4 + 8] = in[1].from;
                }
#pragma unroll
            for (int i = 0; i < KD / 16; ++i) {
                uint32_t s_lo[4];
                split_pair<T>(s[2 * i], s[2 * i + 1], s_hi[i], s_lo);
                sh.state[group][i][0][lane] = as_uint4(s_hi[i]);
                sh.state[group][i][1][lane] = as_uint4(s_lo);
            }
            bar_tell(kBarState + group);
            state_by_rows<T, KD, false>(n, s_hi, s_hi, st.k, lane);
        }
        const float last = row[kDeltaChunk - 1].y;
#pragma unroll
        for (int j = 0; j < KD / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[j][e] *= last;
        float most[2] = {};
        if constexpr (kScaled<T>) {
            rows_largest(s, most);
            most[0] *= in[0].from, most[1] *= in[1].from;
        }
        bar_sync(kBarShare + group);
        // of products with a column of the state that was divided by its power
        auto of = [](float f, const Power &p) { return kScaled<T> ? f * p.from : f; };
        Power by[2];
#pragma unroll
        for (int i = 3; i >= 0; --i) {   // R, and Y = R + (T^ - I) R
            uint32_t v[4], hi[4];
            values_t<VG>(v, st.v[0], i, group, lane);
            float r[2][4];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int j = 2 * i + y;
                const float4 p = sh.ks[group][j][lane];
                const float f0 = row[8 * j + two].y, f1 = row[8 * j + two + 1].y;
                const float2 v0 = widen2<T>(v[2 * y]), v1 = widen2<T>(v[2 * y + 1]);
                r[y][0] = fmaf(-of(f0, in[0]), n[j][0] + p.x, v0.x);
                r[y][1] = fmaf(-of(f1, in[0]), n[j][1] + p.y, v0.y);
                r[y][2] = fmaf(-of(f0, in[1]), n[j][2] + p.z, v1.x);
                r[y][3] = fmaf(-of(f1, in[1]), n[j][3] + p.w, v1.y);
                n[j][0] = r[y][0], n[j][1] = r[y][1], n[j][2] = r[y][2], n[j][3] = r[y][3];
            }
            if constexpr (!kScaled<T>)
                triangle_step<T, false, 2>(n, r[0], r[1], hi, i, st.cell.inverse, lane);
        }
        if constexpr (kScaled<T>)
            triangle_rows<T, false, 2>(n, st.cell.inverse, lane);
        uint32_t hi[4][4], lo[4][4], least[kThree ? 4 : 1][4];
        auto update = [&](float (&u)[4], int j) {   // rows that update the state, as its end has them
            const float4 c0 = row[8 * j + two], c1 = row[8 * j + two + 1];
            const float f0 = c0.z * c0.x, f1 = c1.z * c1.x;
            u[0] = f0 * n[j][0], u[1] = f1 * n[j][1], u[2] = f0 * n[j][2], u[3] = f1 * n[j][3];
        };
        if constexpr (kScaled<T>) {   // they are added to the state: one power for both
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float u[1][4];
                update(u[0], j);
                rows_largest(u, most);
            }
            rows_power<kState>(most, by);
            const float f0 = in[0].from * by[0].to, f1 = in[1].from * by[1].to;
#pragma unroll
            for (int j = 0; j < KD / 8; ++j)
                times_rows(s[j], s[j], f0, f1);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float u[2][4];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int j = 2 * i + y;
                sh.n[group][j][lane] = as_float4(n[j]);
                update(u[y], j);
            }
            if constexpr (kThree)
                split_pair<T>(u[0], u[1], hi[i], lo[i], least[i]);
            else
                split_rows<T>(u[0], u[1], by, hi[i], lo[i]);
        }
        bar_tell(kBarRows + group);
        state_add<T, KD>(s, hi, lo, st.k, lane);
        if constexpr (kScaled<T>)
            in[0] = by[0], in[1] = by[1];
        if constexpr (kThree)
            if (end)
                state_add<T, KD>(s, least, st.k, lane);
    };
    const DeltaTrace trace = SAVE ? a.trace : DeltaTrace();
    const int g16 = (w.v0 >> 4) + group;   // this group of 16 columns among the head's
    constexpr bool kChecked = std::is_same_v<T, __half>;
    bool bad = false;
    auto put_out = [&](typename Shared::Stage &st, int c) {
        const float4 *row = st.cell.row;
        const size_t cell = (size_t)(w.slot + c) * a.HV + w.hv;
        float o[8][4] = {};
        const float score = kScaled<T> ? a.score[cell] : 1.f;   // P's factor
        bar_sync(kBarState + group);
        float in[2] = {1.f, 1.f};
        if constexpr (kScaled<T>)
            in[0] = sh.power[group][lane / 4], in[1] = sh.power[group][lane / 4 + 8];
        {
            uint32_t s_hi[KD / 16][4], s_lo[KD / 16][4];
#pragma unroll
            for (int i = 0; i < KD / 16; ++i)
                take(s_lo[i], sh.state[group][i][1][lane]);
            state_by_rows<T, KD, false>(o, s_lo, s_lo, st.k, lane);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sh.ks[group][j][lane] = as_float4(o[j]);
                o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
            }
            bar_tell(kBarShare + group);
#pragma unroll
            for (int i = 0; i < KD / 16; ++i)
                take(s_hi[i], sh.state[group][i][0][lane]);
            if constexpr (!kScaled<T>)
                if (SAVE && on)
                    put_blocks<KD / 16>(trace.s + cell * trace.s_size, s_hi, 2 * g16, KD / 8, lane);
            state_by_rows<T, KD, true>(o, s_hi, s_lo, st.q, lane);
            if constexpr (SAVE && kScaled<T>) {
                const float most = group_largest(in);
                to_group<KD / 16>(s_hi, in, most);
                if (on) {
                    put_blocks<KD / 16>(trace.s + cell * trace.s_size, s_hi, 2 * g16, KD / 8, lane);
                    if (lane == 0)
                        trace.power[(cell * (a.V / 16) + g16) * 8] = most;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float f0 = row[8 * j + two].w, f1 = row[8 * j + two + 1].w;
            if constexpr (kScaled<T>)
                o[j][0] *= f0 * in[0], o[j][1] *= f1 * in[0], o[j][2] *= f0 * in[1], o[j][3] *= f1 * in[1];
            else
                o[j][0] *= f0, o[j][1] *= f1, o[j][2] *= f0, o[j][3] *= f1;
        }
        bar_sync(kBarRows + group);
        uint32_t hi[4][4];
        if constexpr (kScaled<T>) {
            float n[8][4], p[8][4] = {};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float4 y = sh.n[group][j][lane];
                if (SAVE && on)
                    trace.y[(cell * (a.V / 16) + g16) * 256 + j * 32 + lane] = y;
                const float b0 = row[8 * j + two].x, b1 = row[8 * j + two + 1].x;
                n[j][0] = b0 * y.x, n[j][1] = b1 * y.y, n[j][2] = b0 * y.z, n[j][3] = b1 * y.w;
            }
            Power by[2];
            float largest[2] = {};
            rows_largest(n, largest);
            rows_power<kOperand>(largest, by);
#pragma unroll
            for (int i = 3; i >= 0; --i) {
                times_rows(n[2 * i], n[2 * i], by[0].to, by[1].to);
                times_rows(n[2 * i + 1], n[2 * i + 1], by[0].to, by[1].to);
                triangle_step<T, false, 2, SAVE>(p, n[2 * i], n[2 * i + 1], hi[i], i, st.cell.score, lane);
            }
            const float f0 = score * by[0].from, f1 = score * by[1].from;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                o[j][0] = fmaf(f0, p[j][0], o[j][0]), o[j][1] = fmaf(f0, p[j][1], o[j][1]);
                o[j][2] = fmaf(f1, p[j][2], o[j][2]), o[j][3] = fmaf(f1, p[j][3], o[j][3]);
            }
            if constexpr (SAVE) {
                const float from[2] = {by[0].from, by[1].from}, most = power_of<kTerm>(group_largest(largest)).from;
                to_group<4>(hi, from, most);
                if (on && lane == 0)
                    trace.power[(cell * (a.V / 16) + g16) * 8 + 1] = most;
            }
        } else {
#pragma unroll
            for (int i = 3; i >= 0; --i) {
                float n[2][4];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int j = 2 * i + y;
                    const float4 p = sh.n[group][j][lane];
                    if (SAVE && on)
                        trace.y[(cell * (a.V / 16) + g16) * 256 + j * 32 + lane] = p;
                    const float b0 = row[8 * j + two].x, b1 = row[8 * j + two + 1].x;
                    n[y][0] = b0 * p.x, n[y][1] = b1 * p.y, n[y][2] = b0 * p.z, n[y][3] = b1 * p.w;
                }
                triangle_step<T, false, kThree ? 3 : 2, SAVE>(o, n[0], n[1], hi[i], i, st.cell.score, lane);
            }
        }
        if constexpr (kChecked)
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)   // rows behind the end have q and N of zero
                    bad |= lost(o[j][e]);
        if constexpr (SAVE) {
            if (on)
                put_blocks<4>(trace.n + cell * trace.n_size, hi, 2 * g16, 8, lane);
            float sum[16];   // o.dO of this lane's columns, of rows 8 j + two and + 1
            float most = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t d[4];
                values_t<VG>(d, st.v[1], i, group, lane);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float2 d0 = widen2<T>(d[2 * y]), d1 = widen2<T>(d[2 * y + 1]);
                    if constexpr (kScaled<T>)
                        most = fmaxf(fmaxf(most, fmaxf(fabsf(d0.x), fabsf(d0.y))), fmaxf(fabsf(d1.x), fabsf(d1.y)));
                    const float(&r)[4] = o[2 * i + y];
                    sum[4 * i + 2 * y] = fmaf(r[0], d0.x, r[2] * d1.x);
                    sum[4 * i + 2 * y + 1] = fmaf(r[1], d0.y, r[3] * d1.y);
                }
            }
            if constexpr (kScaled<T>) {
                most = warp_largest(most);
                if (on && lane == 0)
                    trace.power[(cell * (a.V / 16) + g16) * 8 + 2] = power_of<kTerm>(most).from;
            }
            // over the eight lanes of a row pair: of the 16 sums each lane is left with two, rows of tile lane / 4
            sum_over_columns<16>(sum, lane);
            if (on)
                *reinterpret_cast<float2 *>(trace.dots + ((cell * (a.V / 16) + g16) * 3) * 64 + 8 * (lane / 4) + two) = make_float2(sum[0], sum[1]);
        } else {
            const int rows = min(kDeltaChunk, w.len - c * kDeltaChunk);
            To *out = static_cast<To *>(a.o) + (((size_t)w.bos + (size_t)c * kDeltaChunk) * a.HV + w.hv) * a.V + col;
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = 8 * j + two + (e & 1);
                    if (on && t < rows)
                        out[(size_t)t * a.HV * a.V + (e >> 1) * 8] = narrow<To>(o[j][e]);
                }
        }
    };

    // the warps of a role go their own ways through a chunk and meet at its end
    auto walk = [&](auto work) {
        if (tid == kThreads / 2 && w.chunks)
            ask_chunk(a, maps, w, sh, 0, 0, kCell, 0);
        for (int c = 0; c < w.chunks; ++c) {
            const bool ok = tc::bar_wait(&sh.full[c & 1], (c >> 1) & 1);
            if (__syncthreads_or(!ok)) {
                give_up(a.status, &sh.full[c & 1], (c >> 1) & 1);
                return;
            }
            if (tid == kThreads / 2 && c + 1 < w.chunks)
                ask_chunk(a, maps, w, sh, c + 1, c + 1, kCell, 0);
            if (w.len - c * kDeltaChunk < kDeltaChunk) {
                clear_tail<VG>(sh.stage[c & 1], w.len - c * kDeltaChunk);
                __syncthreads();
            }
            work(sh.stage[c & 1], c);
        }
    };
    if (!output) {
        float s[KD / 8][4];
        state_io<KD>(s, nullptr, a.h0, state, a.V, col, on, false);
        if constexpr (kScaled<T>) {
            rows_power<kState>(s, in);
#pragma unroll
            for (int j = 0; j < KD / 8; ++j)
                times_rows(s[j], s[j], in[0].to, in[1].to);
        }
        walk([&](auto &st, int c) {
            chain(st, s, c + 1 == w.chunks);
            if (SAVE && on && ((c + 1) % kDeltaKept == 0 || c + 1 == w.chunks)) {
                float4 *to = a.trace.kept + delta_kept_at(a, w.n, c, w.hv, g16) * (KD / 8 * 32) + lane;
#pragma unroll
                for (int j = 0; j < KD / 8; ++j) {
                    float r[4] = {s[j][0], s[j][1], s[j][2], s[j][3]};
                    if constexpr (kScaled<T>)
                        times_rows(r, r, in[0].from, in[1].from);
                    to[j * 32] = as_float4(r);
                }
            }
        });
        if constexpr (kScaled<T>)
#pragma unroll
            for (int j = 0; j < KD / 8; ++j)
                times_rows(s[j], s[j], in[0].from, in[1].from);
        report_lost<T>(a, s, false);
        if (!SAVE && a.ht)
            state_io<KD>(s, a.ht, nullptr, state, a.V, col, on, true);
    } else {
        walk([&](auto &st, int c) { put_out(st, c); });
        if (kChecked && bad)
            report(a.status, GLA_ERR_RANGE);
    }
}

}  // namespace

cudaError_t launch_delta_chain(const DeltaArgs &a, int dtype, bool save, cudaStream_t s)
{
    return delta_types(dtype, [&](auto x, auto o) {
        typedef std::remove_pointer_t<decltype(x)> T;
        typedef std::remove_pointer_t<decltype(o)> To;
        if constexpr (std::is_same_v<T, float>) {
            return cudaErrorInvalidValue;
        } else {
            auto go = [&](auto kd, auto vg) {
                constexpr int KD = decltype(kd)::value, VG = decltype(vg)::value;
                constexpr bool kHalf = std::is_same_v<T, __half>;
                if (!save)
                    return launch_chain(delta_chain_kernel<T, To, KD, VG, false>, sizeof(ChainShared<KD, VG, 1, DeltaCell>), VG, kHalf, a, s);
                if constexpr (std::is_same_v<To, float>)   // the gradients' pass has no output of another type
                    return launch_chain(delta_chain_kernel<T, float, KD, VG, true>, sizeof(ChainShared<KD, VG, 2, DeltaCell>), VG, kHalf, a, s);
                else
                    return cudaErrorInvalidValue;
            };
            auto by_keys = [&](auto vg) { return a.K == 128 ? go(Int<128>(), vg) : go(Int<64>(), vg); };
            return few_columns(a) ? by_keys(Int<2>()) : by_keys(Int<4>());
        }
    });
}

}  // namespace gla
