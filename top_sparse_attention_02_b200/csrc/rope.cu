// rope.cu -- the two ends of a decode step around its attention: queries and
// keys made (RMS norm of each head, position rotation), and new keys and values
// put into a paged cache (keys rotated on the way).
//
// Per head of 128 elements:
//   y = x / sqrt(mean(x^2) + eps) * w                          (w given)
//   pairs (a, b) of the first rot_dim elements -> (a cos t - b sin t,
//   b cos t + a sin t), t = position * inv_freq[i], the pair i being
//   (i, i + rot_dim/2), or (2i, 2i + 1) when interleaved.
//
// Both are streams: each element is read once and written once, with about ten
// operations between, so HBM bounds long calls and the launch bounds short
// ones.  A half-warp holds a head (16 bytes a lane): the norm's sum is four
// shuffles, and a lane's rotation partners are all in one other lane (rot_dim is
// a multiple of 16), so no element passes through shared memory.  The angles are
// the costly part (a 64-bit product each, since position * inv_freq loses its
// fraction in 32 bits at far positions, then a sine and a cosine): each CTA
// computes them once per token into shared memory and every head of the token
// uses them.
#include <cuda_fp16.h>

#include "common.cuh"
#include "paged.cuh"

namespace tsa {

constexpr int kRopeThreads = 256;
constexpr int kRopeHalfWarps = kRopeThreads / 16;
constexpr int kRopeMaxTokens = 4;  // tokens of one CTA

// cos and sin of position * inv_freq.  The product in turns is reduced to
// [-1/2, 1/2] in 64 bits, where positions up to 2^31 keep 20 bits of fraction or more.
__device__ __forceinline__ float2 rope_angle(int pos, double inv_freq) {
    double turns = (double)pos * (inv_freq * 0.15915494309189533577);  // 1 / (2 pi)
    turns -= rint(turns);
    float s, c;
    sincospif(2.0f * (float)turns, &s, &c);
    return make_float2(c, s);
}

struct RopeTile {
    float2 cs[kRopeMaxTokens][kD / 2];
};

// the CTA's angles: token i of tok positions pos(i)
template <class Pos>
__device__ __forceinline__ void rope_angles(RopeTile& s, int ntok, const Rotation& rot, Pos pos) {
    const int half = rot.rot_dim >> 1;
    for (int j = threadIdx.x; j < ntok * half; j += kRopeThreads) {
        const int i = j / half, f = j - i * half;
        s.cs[i][f] = rope_angle(pos(i), rot.inv_freq[f]);
    }
}

// this lane's angles of one token: x[j] -> x[j] * c[j] + partner * s[j]
struct LaneRot {
    float c[8], s[8];
    int src;       // split pairs: the lane (of 32) that holds the partners
    bool on;       // this lane's elements are rotated
    __device__ __forceinline__ void load(const float2* cs, const Rotation& rot, int lane) {
        const int l = lane & 15, h = rot.rot_dim >> 4;
        on = l < 2 * h;
        src = lane;
        if (!on) return;
        if (rot.interleaved) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 v = cs[l * 4 + j];
                c[2 * j] = c[2 * j + 1] = v.x;
                s[2 * j] = -v.y;
                s[2 * j + 1] = v.y;
            }
        } else {
            const bool low = l < h;
            src = low ? lane + h : lane - h;
            const int i0 = (low ? l : l - h) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 v = cs[i0 + j];
                c[j] = v.x;
                s[j] = low ? -v.y : v.y;
            }
        }
    }
    // all 32 lanes call this together
    __device__ __forceinline__ void apply(float (&x)[8], bool interleaved) const {
        if (interleaved) {
            if (!on) return;
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float a = x[j], b = x[j + 1];
                x[j] = fmaf(b, s[j], a * c[j]);
                x[j + 1] = fmaf(a, s[j + 1], b * c[j + 1]);
            }
            return;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float p = __shfl_sync(0xffffffffu, x[j], src);
            if (on) x[j] = fmaf(p, s[j], x[j] * c[j]);
        }
    }
};

template <class E>
__global__ void __launch_bounds__(kRopeThreads)
qk_norm_rope_kernel(Heads q, Heads k, Heads qo, Heads ko, int T, int Hq, int Hkv, const float* __restrict__ wq,
                    const float* __restrict__ wk, float eps, const int32_t* __restrict__ positions, Rotation rot,
                    int tok_cta) {
    __shared__ RopeTile s;
    griddep_wait();
    const int t0 = blockIdx.x * tok_cta, ntok = min(tok_cta, T - t0);
    const int lane = threadIdx.x & 31, l = lane & 15;
    // half-warps of one token: 16 / tok_cta, a power of two
    const int per = kRopeHalfWarps / tok_cta, hw = threadIdx.x >> 4;
    const int i = hw / per, first = hw - i * per;
    const int t = t0 + i;
    const bool live = i < ntok;
    const int H = Hq + Hkv;
    auto src = [&](int h) {
        return h < Hq ? static_cast<const uint16_t*>(q.p) + t * q.st + h * q.sh
                      : static_cast<const uint16_t*>(k.p) + t * k.st + (h - Hq) * k.sh;
    };
    constexpr int U = 4;  // heads in flight per half-warp
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = first + u * per;
        if (live && h < H) raw[u] = *reinterpret_cast<const uint4*>(src(h) + l * 8);
    }
    LaneRot lr;
    lr.on = false;
    lr.src = lane;
    if (rot.rot_dim > 0) {
        rope_angles(s, ntok, rot, [&](int j) { return positions[t0 + j]; });
        __syncthreads();
        if (live) lr.load(s.cs[i], rot, lane);
    }
    const int steps = (H + per - 1) / per;  // the same for every half-warp: the shuffles below need all lanes
    for (int n = 0; n < steps; n += U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = first + (n + u) * per;
            const bool act = live && h < H;
            float x[8] = {};
            if (act) E::unpack8(raw[u], x);
            const int hn = h + U * per;
            if (live && hn < H) raw[u] = *reinterpret_cast<const uint4*>(src(hn) + l * 8);
            const float* w = h < Hq ? wq : wk;
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
            for (int m = 1; m < 16; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
            if (w) {
                const float r = 1.0f / sqrtf(ss * (1.0f / kD) + eps);
                const float4 w0 = *reinterpret_cast<const float4*>(w + l * 8);
                const float4 w1 = *reinterpret_cast<const float4*>(w + l * 8 + 4);
                const float wv[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = x[j] * r * wv[j];
            }
            lr.apply(x, rot.interleaved);
            if (act) {
                uint16_t* dst = h < Hq ? static_cast<uint16_t*>(const_cast<void*>(qo.p)) + t * qo.st + h * qo.sh
                                       : static_cast<uint16_t*>(const_cast<void*>(ko.p)) + t * ko.st + (h - Hq) * ko.sh;
                *reinterpret_cast<uint4*>(dst + l * 8) = E::pack8(x);
            }
        }
    }
    griddep_launch();
}

template <class E>
__global__ void __launch_bounds__(kRopeThreads)
paged_append_kernel(Pages c, Heads k, Heads v, int T, const int32_t* __restrict__ seq, const int32_t* __restrict__ row,
                    const int32_t* __restrict__ positions, Rotation rot, unsigned* __restrict__ flag, int tok_cta) {
    __shared__ RopeTile s;
    griddep_wait();
    const int t0 = blockIdx.x * tok_cta, ntok = min(tok_cta, T - t0);
    const int lane = threadIdx.x & 31, l = lane & 15;
    const int per = kRopeHalfWarps / tok_cta, hw = threadIdx.x >> 4;
    const int i = hw / per, first = hw - i * per;
    const int t = t0 + i;
    // where the token goes: a negative sequence is padding (skipped), anything
    // else out of range sets the flag and is skipped
    long long at = -1;
    if (i < ntok) {
        const int b = seq ? seq[t] : t, r = row[t];
        if (b >= c.B || (b >= 0 && (r < 0 || r >= c.rows_cap()))) {
            if (first == 0 && l == 0) atomicOr(flag, kFlagBounds);
        } else if (b >= 0) {
            const int pg = r / c.page_size;
            const int page = c.table[(long long)b * c.width + pg];
            if (page < 0 || page >= c.num_pages) {
                if (first == 0 && l == 0) atomicOr(flag, kFlagBounds);
            } else {
                at = page * c.page_stride + (long long)(r - pg * c.page_size) * c.row_stride;
            }
        }
    }
    const bool live = at >= 0;
    LaneRot lr;
    lr.on = false;
    lr.src = lane;
    if (rot.rot_dim > 0) {
        const int32_t* ps = positions ? positions : row;
        rope_angles(s, ntok, rot, [&](int j) { return ps[t0 + j]; });
        __syncthreads();
        if (live) lr.load(s.cs[i], rot, lane);
    }
    const int H = 2 * c.Hkv, steps = (H + per - 1) / per;
    for (int n = 0; n < steps; ++n) {
        const int h = first + n * per;
        const bool act = live && h < H, is_k = h < c.Hkv;
        const int hh = is_k ? h : h - c.Hkv;
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (act)
            raw = *reinterpret_cast<const uint4*>(is_k ? static_cast<const uint16_t*>(k.p) + t * k.st + hh * k.sh + l * 8
                                                       : static_cast<const uint16_t*>(v.p) + t * v.st + hh * v.sh + l * 8);
        // a value head, or an unrotated lane of a key head, is copied bit by bit
        float x[8];
        E::unpack8(raw, x);
        lr.apply(x, rot.interleaved);
        if (act) {
            uint16_t* dst = static_cast<uint16_t*>(is_k ? c.K : c.V) + at + hh * c.head_stride + l * 8;
            *reinterpret_cast<uint4*>(dst) = is_k && lr.on ? E::pack8(x) : raw;
        }
    }
    griddep_launch();
}

// tokens of one CTA: four when that still gives every SM two CTAs (each token's
// angles then cost a quarter of a CTA's set-up), else one
static int rope_tokens(int T) { return T >= 4 * 2 * kPagedSms ? kRopeMaxTokens : 1; }

template <class... P, class... A>
static cudaError_t rope_launch(void (*kernel)(P...), int T, cudaStream_t st, int tok, A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((T + tok - 1) / tok));
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1] = {pdl_attr()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
    note_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_qk_norm_rope(const Heads& q, const Heads& k, const Heads& qo, const Heads& ko, int T, int Hq, int Hkv,
                                int half, const float* q_weight, const float* k_weight, float eps,
                                const int32_t* positions, const Rotation& rot, cudaStream_t st) {
    if (T == 0 || Hq + Hkv == 0) return cudaSuccess;
    const int tok = rope_tokens(T);
    return rope_launch(half ? qk_norm_rope_kernel<F16> : qk_norm_rope_kernel<Bf16>, T, st, tok, q, k, qo, ko, T, Hq, Hkv,
                       q_weight, k_weight, eps, positions, rot, tok);
}

cudaError_t launch_paged_append(const Pages& c, const Heads& k, const Heads& v, int T, const int32_t* seq,
                                const int32_t* row, const int32_t* positions, const Rotation& rot, unsigned* flag,
                                cudaStream_t st) {
    if (T == 0) return cudaSuccess;
    const int tok = rope_tokens(T);
    return rope_launch(c.half ? paged_append_kernel<F16> : paged_append_kernel<Bf16>, T, st, tok, c, k, v, T, seq, row,
                       positions, rot, flag, tok);
}

}  // namespace tsa
