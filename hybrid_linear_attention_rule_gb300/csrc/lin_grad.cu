// lin_grad.cu -- linear attention's prefill and gradients as jobs (lin.cuh), and the gradient of the decays.
//
// The gradient of g_t is what passes over it: f(t) = sum over s < t <= u of e^{G_u - G_s} (q_u . k_s) (do_u . v_s) scale, with
// the first state as a token before the first and the last state's gradient as one behind the last.  f(t) - f(t + 1) =
// r1_t - r2_t, r1 the pairs that end at t (q_t . dq_t without s = t), r2 those that begin there (v_t . dv_t without u = t): the
// jobs write both.  Summed from the sequence's end alone, the rounding of every later token would stay in f(t); so at anchors,
// every 512 tokens, f is worked out directly as <S, R> of the two states that the jobs left there, and the sums, in 64
// bits, start anew.  Where a sum from an anchor behind is not finite, that from the anchor before is taken, if it is.  Leaving the pairs s = t = u out keeps them from cancelling where the decay is strong.
#include <algorithm>

#include "lin.cuh"

namespace k3kda {
namespace lin {
namespace {

// f at the anchors: <S, R> with S [dv, dk] and R [dk, dv].  A CTA for each (anchor, head), a thread blocks of 4 by 4 of both, whose
// pieces of 16 bytes fill whole lines of S and whole sectors of R; products of FP32, eight of them summed in FP32, the rest in 64 bits.  HBM
// bounds it: 67 MB for 8 k tokens and 32 heads in 16 us, where reads of S
// down its columns took 39.  (S laid out as R by the job that leaves it: its
// scattered stores held its chunks up, 311 to 404 us.)
struct AnchorArgs {
    const float *S, *R, *dlast;       // dlast [N, H, dk, dv] or null
    double *f;                        // [slots, H]
    const int32_t *cu;
    int N, T, H, dk, dv;
};

__global__ void __launch_bounds__(256) anchor_kernel(const __grid_constant__ AnchorArgs A) {
    __shared__ double part[8];
    const int h = blockIdx.y, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int across = (A.dk + 31) / 32, tiles = across * (A.dv / 16);
    for (int n = blockIdx.x; n < A.N; n += gridDim.x) {
        int begin, end;
        seq_bounds(A.cu, n, A.T, begin, end);
        const int count = max(1, (end - begin + kAnchor - 1) / kAnchor);
        for (int k = blockIdx.z; k < count; k += gridDim.z) {
            const size_t at = (size_t)(anchor_slot(begin, n) + k) * A.H + h;
            const bool last = k == count - 1;
            const float *R = last ? (A.dlast ? A.dlast + ((size_t)n * A.H + h) * A.dk * A.dv : nullptr) : A.R + at * A.dk * A.dv;
            double sum = 0.0;
            if (R) {
                const float *S = A.S + at * A.dk * A.dv;
#pragma unroll 2
                for (int tile = warp; tile < tiles; tile += 8) {
                    const int i0 = tile % across * 32 + lane % 8 * 4, j0 = tile / across * 16 + lane / 8 * 4;
                    if (i0 >= A.dk) continue;
                    float4 s[4], r[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        s[u] = __ldg(reinterpret_cast<const float4 *>(S + (size_t)(j0 + u) * A.dk + i0));
                        r[u] = __ldg(reinterpret_cast<const float4 *>(R + (size_t)(i0 + u) * A.dv + j0));
                    }
                    const float a = fmaf(s[0].x, r[0].x, fmaf(s[1].x, r[0].y, fmaf(s[2].x, r[0].z, s[3].x * r[0].w)));
                    const float b = fmaf(s[0].y, r[1].x, fmaf(s[1].y, r[1].y, fmaf(s[2].y, r[1].z, fmaf(s[3].y, r[1].w, a))));
                    const float c = fmaf(s[0].z, r[2].x, fmaf(s[1].z, r[2].y, fmaf(s[2].z, r[2].z, s[3].z * r[2].w)));
                    const float d = fmaf(s[0].w, r[3].x, fmaf(s[1].w, r[3].y, fmaf(s[2].w, r[3].z, fmaf(s[3].w, r[3].w, c))));
                    sum += b;
                    sum += d;
                }
                for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            }
            if (lane == 0) part[warp] = sum;
            __syncthreads();
            if (threadIdx.x == 0) {
                sum = 0.0;
                for (int u = 0; u < 8; ++u) sum += part[u];
                A.f[at] = sum;
            }
            __syncthreads();
        }
    }
}

// dg: a CTA sums one stretch between anchors for 8 heads (a 32-byte piece of a row), 64 runs of 8 tokens, each a thread a head.  The runs
// behind a thread's own come by shuffles (a warp has four) and one sum a warp, so that few additions are in 64 bits, of which an SM
// does about two a cycle; a run's own eight are in FP32, as its terms are.  8 k tokens of 32 heads (8 MB): 11 us, 15 with those in
// 64 bits too; 5 sequences to 1,900 tokens of 16 heads 10.6 us, 24 then and with their stretches one after the other.
struct SumArgs {
    const float *r1, *r2;             // [slices][T, H]
    int n1, n2;                       // slices
    const double *f;
    float *dg;                        // [T, H]
    const int32_t *cu;
    int N, T, H;
    const float *first, *dfirst, *R;  // [N, H, dk, dv] or null; R's anchors, which hold the first state's gradient where `dfirst` does not
    int dk, dv;
};

// The same stretch from its beginning on, f(t + 1) = f(t) - (r1_t - r2_t), for the tokens whose sum from the end is not finite: a key or value
// that is not reaches the anchor behind it and its own r2, but no f(t) up to its token.  (A query or an output's gradient that is not
// reaches no f(t) behind its token, where the sums from the end hold.)  Rare, so simple: sums of all in 64 bits.
__device__ __noinline__ void sum_from_begin(const SumArgs &A, int n, int k, int begin, int end) {
    __shared__ double room[64][8];
    const int hl = threadIdx.x % 8, run = threadIdx.x / 8, h = blockIdx.y * 8 + hl;
    const int t0 = min(begin + k * kAnchor + run * 8, end), t1 = min(t0 + 8, end);
    const size_t TH = (size_t)A.T * A.H;
    const long long slot = anchor_slot(begin, n);
    auto step = [&](int t) {
        double d = 0.0;
        for (int u = 0; u < A.n1; ++u) d += A.r1[u * TH + (size_t)t * A.H + h];
        for (int u = 0; u < A.n2; ++u) d -= A.r2[u * TH + (size_t)t * A.H + h];
        return d;
    };
    // f at the stretch's first token: the anchor before, or <first state, its gradient>
    double f = 0.0;
    if (k == 0 && A.first && h < A.H) {
        const size_t size = (size_t)A.dk * A.dv, at = ((size_t)n * A.H + h) * size;
        const float *S = A.first + at, *R = A.dfirst ? A.dfirst + at : A.R + ((size_t)(slot + (end - begin - 1) / kAnchor) * A.H + h) * size;
        for (size_t i = run; i < size; i += 64) f += (double)S[i] * R[i];
    }
    room[run][hl] = f;
    __syncthreads();
    f = 0.0;
    if (k > 0 && h < A.H) f = A.f[(size_t)(slot + k - 1) * A.H + h];
    else
        for (int u = 0; u < 64; ++u) f += room[u][hl];
    __syncthreads();
    double all = 0.0;
    if (h < A.H)
        for (int t = t0; t < t1; ++t) all += step(t);
    room[run][hl] = all;
    __syncthreads();
    for (int u = 0; u < run; ++u) f -= room[u][hl];
    if (h < A.H)
        for (int t = t0; t < t1; ++t) {
            float &to = A.dg[(size_t)t * A.H + h];
            if (!isfinite(to) && isfinite((float)f)) to = (float)f;
            f -= step(t);
        }
    __syncthreads();
}

__global__ void __launch_bounds__(512) sum_kernel(const __grid_constant__ SumArgs A) {
    constexpr int RUN = 8;
    static_assert(kAnchor == RUN * 64, "512 threads, 8 of them a run");
    __shared__ double part[16][8];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, hl = threadIdx.x % 8, run = threadIdx.x / 8, h = blockIdx.y * 8 + hl;
    const size_t TH = (size_t)A.T * A.H;
    bool lost = false;                                               // a sum of the thread's that is not finite
    for (int n = blockIdx.x; n < A.N; n += gridDim.x) {
        int begin, end;
        seq_bounds(A.cu, n, A.T, begin, end);
        const int count = (end - begin + kAnchor - 1) / kAnchor;
        for (int k = blockIdx.z; k < count; k += gridDim.z) {
            const int t0 = begin + k * kAnchor + run * RUN, t1 = min(t0 + RUN, end);
            float p[RUN], q[RUN];
#pragma unroll
            for (int i = 0; i < RUN; ++i) p[i] = q[i] = 0.f;
            if (h < A.H) {
#pragma unroll 4
                for (int u = 0; u < A.n1; ++u)
#pragma unroll
                    for (int i = 0; i < RUN; ++i)
                        if (t0 + i < t1) p[i] += A.r1[u * TH + (size_t)(t0 + i) * A.H + h];
#pragma unroll 4
                for (int u = 0; u < A.n2; ++u)
#pragma unroll
                    for (int i = 0; i < RUN; ++i)
                        if (t0 + i < t1) q[i] += A.r2[u * TH + (size_t)(t0 + i) * A.H + h];
            }
            // the run's own sums, from each token to its end
            p[RUN - 1] -= q[RUN - 1];
#pragma unroll
            for (int i = RUN - 2; i >= 0; --i) p[i] = p[i + 1] + (p[i] - q[i]);
            const double sum = p[0];
            // of the warp's runs: those from the thread's own on, those behind it
            const double next = __shfl_down_sync(0xffffffffu, sum, 8), pair = lane < 24 ? sum + next : sum;
            const double far = __shfl_down_sync(0xffffffffu, pair, 16), from = lane < 16 ? pair + far : pair;
            const double after = __shfl_down_sync(0xffffffffu, from, 8);
            if (lane < 8) part[warp][lane] = from;
            __syncthreads();
            if (h < A.H) {
                double f = A.f[(size_t)(anchor_slot(begin, n) + k) * A.H + h];
                for (int u = 15; u > warp; --u) f += part[u][hl];
                if (lane < 24) f += after;
                const float whole = (float)f, rest = (float)(f - whole);
#pragma unroll
                for (int i = 0; i < RUN; ++i)
                    if (t0 + i < t1) {
                        const float v = whole + (rest + p[i]);
                        lost = lost || !isfinite(v);
                        A.dg[(size_t)(t0 + i) * A.H + h] = v;
                    }
            }
            __syncthreads();
        }
    }
    // (behind the loops, whose registers a call within them would spill)
    if (__syncthreads_or(lost))
        for (int n = blockIdx.x; n < A.N; n += gridDim.x) {
            int begin, end;
            seq_bounds(A.cu, n, A.T, begin, end);
            const int count = (end - begin + kAnchor - 1) / kAnchor;
            for (int k = blockIdx.z; k < count; k += gridDim.z) sum_from_begin(A, n, k, begin, end);
        }
}

// One decay a head for all tokens: its gradient is the sum over them, in 64 bits and in a fixed order.  A CTA a head.
__global__ void __launch_bounds__(512) fixed_kernel(const float *dg, float *out, const int32_t *cu, int N, int T, int H) {
    __shared__ double part[16];
    const int h = blockIdx.x;
    double sum = 0.0;
    for (int n = 0; n < N; ++n) {
        int begin, end;
        seq_bounds(cu, n, T, begin, end);
        for (int t = begin + (int)threadIdx.x; t < end; t += 512) sum += dg[(size_t)t * H + h];
    }
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        sum = 0.0;
        for (int u = 0; u < 16; ++u) sum += part[u];
        out[h] = (float)sum;
    }
}

// Gradients of shared heads: out[t, hk, c] = sum over its group of part[t, h, c], rounded once.  Tokens of no sequence are left alone.  A stream:
// HBM or, for short calls, a launch's latency bounds it.
__global__ void __launch_bounds__(256) group_kernel(const float *p1, const float *p2, void *o1, void *o2, int bf16, const int32_t *cu, int N, int T,
                                                    int Hk, int group, int d) {
    const int n = blockIdx.z;
    int begin, end;
    seq_bounds(cu, n, T, begin, end);
    const float *part = blockIdx.y ? p2 : p1;
    void *out = blockIdx.y ? o2 : o1;
    const size_t row = (size_t)Hk * (d / 4), i0 = begin * row, i1 = end * row;
    for (size_t i = i0 + blockIdx.x * 256 + threadIdx.x; i < i1; i += (size_t)gridDim.x * 256) {
        const size_t head = i / (d / 4), c = i % (d / 4) * 4;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int u = 0; u < group; ++u) {
            const float4 v = *reinterpret_cast<const float4 *>(part + (head * group + u) * d + c);
            s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
        }
        if (bf16) {
            __nv_bfloat162 r[2] = {__floats2bfloat162_rn(s.x, s.y), __floats2bfloat162_rn(s.z, s.w)};
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(out) + head * d + c) = *reinterpret_cast<uint2 *>(r);
        } else {
            *reinterpret_cast<float4 *>(static_cast<float *>(out) + head * d + c) = s;
        }
    }
}

size_t round256(size_t b) { return (b + 255) & ~size_t(255); }

// The workspace: the status word, the states of the pieces that sequences are cut into, and the gradient's parts.
struct Space {
    size_t pieces, r1, r2, S, R, f, dg, pq, pk, total;
    Space(int N, int T, int Hk, int H, int dk, int dv, int bf16, bool backward) {
        size_t at = 256;
        auto take = [&](size_t bytes) {
            const size_t was = at;
            at += round256(bytes);
            return was;
        };
        const size_t TH = (size_t)T * H, slots = anchor_slots(N, T);
        const int width = slice_width(N, T, H, 3, dk > dv ? dk : dv);
        pieces = take(bf16 ? tc_workspace(N, T, H, backward ? 2 : 1) : f32_workspace());
        r1 = r2 = S = R = f = dg = pq = pk = at;
        if (backward) {
            r1 = take(TH * (bf16 ? 4 : slices(dk, width)) * 4);
            r2 = take(TH * (bf16 ? 4 : slices(dv, width)) * 4);
            S = take(slots * H * dk * dv * 4);
            R = take(slots * H * dk * dv * 4);
            f = take(slots * H * 8);
            dg = take(TH * 4);
            if (H > Hk) {
                pq = take(TH * dk * 4);
                pk = take(TH * dk * 4);
            }
        }
        total = at;
    }
};

Call call_of(const LinArgs &a, const Space &w) {
    Call c{};
    c.bf16 = a.bf16;
    c.g = a.g;
    c.fixed = a.fixed;
    c.cu = a.cu;
    c.N = a.N;
    c.T = a.T;
    c.H = a.H;
    c.slot = a.slot;
    c.num_slots = a.num_slots;
    c.status = static_cast<unsigned *>(a.ws);
    c.pieces = static_cast<char *>(a.ws) + w.pieces;
    return c;
}

bool on_tensor_cores(const Call &c) { return c.bf16 && c.T > 0; }
cudaError_t launch_scan(const Call &c, bool apart, cudaStream_t s) { return on_tensor_cores(c) ? launch_scan_tc(c, apart, s) : launch_scan_f32(c, s); }

}  // namespace
}  // namespace lin

using namespace lin;

size_t lin_workspace(int N, int T, int Hk, int H, int dk, int dv, int bf16, int backward) {
    return Space(N, T, Hk, H, dk, dv, bf16, backward != 0).total;
}

cudaError_t launch_lin_prefill(const LinArgs &a, void *out, int out_bf16, float *last, cudaStream_t s) {
    const Space w(a.N, a.T, a.Hk, a.H, a.dk, a.dv, a.bf16, false);
    const int group = a.H / a.Hk;
    Call c = call_of(a, w);
    c.jobs = 1;
    Job &j = c.job[0];
    j.x = {a.q, group};
    j.y = {a.k, group};
    j.z = {a.v, 1};
    j.a = a.dk;
    j.b = a.dv;
    j.sp = j.sc = a.scale;
    j.sw = 1.f;
    j.first = a.first;
    j.last = last;
    j.sa = a.dv;
    j.sb = 1;
    j.out = out;
    j.out_bf16 = out_bf16;
    j.exact = !out_bf16;
    return launch_scan(c, false, s);
}

cudaError_t launch_lin_backward(const LinArgs &a, const void *dO, const float *dlast, void *dq, void *dk, void *dv, float *dg,
                                float *dfirst, cudaStream_t s) {
    const Space w(a.N, a.T, a.Hk, a.H, a.dk, a.dv, a.bf16, true);
    const int group = a.H / a.Hk;
    char *ws = static_cast<char *>(a.ws);
    auto part = [&](size_t at) { return reinterpret_cast<float *>(ws + at); };
    Call c = call_of(a, w);
    c.jobs = 3;
    Job &jq = c.job[0], &jv = c.job[1], &jk = c.job[2];
    jq.x = {dO, 1};
    jq.y = {a.v, 1};
    jq.z = {a.k, group};
    jq.a = a.dv;
    jq.b = a.dk;
    jq.sp = jq.sc = a.scale;
    jq.sw = 1.f;
    jq.first = a.first;
    jq.sa = 1;
    jq.sb = a.dv;
    jv.x = {a.k, group};
    jv.y = {a.q, group};
    jv.z = {dO, 1};
    jv.a = a.dk;
    jv.b = a.dv;
    jv.reverse = 1;
    jv.sp = jv.sw = a.scale;
    jv.sc = 1.f;
    jv.first = dlast;
    jv.last = dfirst;
    jv.sa = a.dv;
    jv.sb = 1;
    jk.x = {a.v, 1};
    jk.y = {dO, 1};
    jk.z = {a.q, group};
    jk.a = a.dv;
    jk.b = a.dk;
    jk.reverse = 1;
    jk.sp = jk.sw = a.scale;
    jk.sc = 1.f;
    jk.first = dlast;
    jk.sa = 1;
    jk.sb = a.dv;
    // gradients of shared heads are summed in FP32 first
    jq.out = group > 1 ? part(w.pq) : dq;
    jk.out = group > 1 ? part(w.pk) : dk;
    jv.out = dv;
    jq.out_bf16 = jk.out_bf16 = group > 1 ? 0 : a.bf16;
    jv.out_bf16 = a.bf16;
    if (dg) {
        jq.r = {a.q, group};
        jq.dots = part(w.r1);
        jq.anchors = part(w.S);
        jq.last_anchor = dlast != nullptr;
        jq.exact = 1;
        jv.r = {a.v, 1};
        jv.dots = part(w.r2);
        jv.anchors = part(w.R);
        jv.last_anchor = a.first && !dfirst;
        jv.exact = 1;
    }
    if (cudaError_t e = launch_scan(c, dg != nullptr, s)) return e;
    const unsigned seqs = (unsigned)(a.N < 1024 ? a.N : 1024);
    if (dg) {
        // stretches between anchors that CTAs take at once: all, unless these are many
        auto deep = [&](int across) {
            const unsigned mean = a.T / kAnchor / seqs + 1, room = 1024 / (seqs * across), most = a.T / kAnchor + 1;
            return std::min(std::min(std::max(mean, room), most), 256u);
        };
        double *f = reinterpret_cast<double *>(ws + w.f);
        const AnchorArgs g{part(w.S), part(w.R), dlast, f, a.cu, a.N, a.T, a.H, a.dk, a.dv};
        anchor_kernel<<<dim3(seqs, a.H, deep(a.H)), 256, 0, s>>>(g);
        if (cudaError_t e = launched()) return e;
        float *to = a.fixed ? part(w.dg) : dg;
        const int width = slice_width(a.N, a.T, a.H, c.jobs, a.dk > a.dv ? a.dk : a.dv);
        const SumArgs u{part(w.r1), part(w.r2), on_tensor_cores(c) ? 4 : slices(a.dk, width), on_tensor_cores(c) ? 4 : slices(a.dv, width), f, to, a.cu, a.N, a.T, a.H,
                        a.first, dfirst, part(w.R), a.dk, a.dv};
        sum_kernel<<<dim3(seqs, (a.H + 7) / 8, deep((a.H + 7) / 8)), 512, 0, s>>>(u);
        if (cudaError_t e = launched()) return e;
        if (a.fixed) {
            fixed_kernel<<<a.H, 512, 0, s>>>(to, dg, a.cu, a.N, a.T, a.H);
            if (cudaError_t e = launched()) return e;
        }
    }
    if (group > 1) {
        const size_t rows = (size_t)a.T * a.Hk * (a.dk / 4) / a.N / 256 + 1;
        for (int n = 0; n < a.N; n += 65535) {
            const int here = a.N - n < 65535 ? a.N - n : 65535;
            group_kernel<<<dim3((unsigned)(rows < 2048 ? rows : 2048), 2, here), 256, 0, s>>>(part(w.pq), part(w.pk), dq, dk, a.bf16,
                                                                                            a.cu ? a.cu + n : nullptr, here, a.T, a.Hk, group, a.dk);
            if (cudaError_t e = launched()) return e;
        }
    }
    return cudaSuccess;
}

}  // namespace k3kda
