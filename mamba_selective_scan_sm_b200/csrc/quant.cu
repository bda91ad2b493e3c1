// Launches of the 8-bit kernels and their C ABI (include/ssm.h).
#define SSM_ERROR_WORD g_error_quant
#include "quant_kernel.cuh"

#include <type_traits>

#include "api_common.h"

namespace ssm {

cudaError_t launch_pack(int elem_size, bool channel_last, const PackParams& p, cudaStream_t st) {
    const int nb = (p.seqlen + kBlock8 - 1) / kBlock8;
    if (channel_last) {
        const dim3 g((p.dim + 255) / 256, nb < 65535 ? nb : 65535, p.batch);
        if (elem_size == 2) pack_cl_kernel<__nv_bfloat16><<<g, 256, 0, st>>>(p);
        else pack_cl_kernel<float><<<g, 256, 0, st>>>(p);
    } else {
        const int64_t threads = (int64_t)p.batch * p.dim * nb * 8;
        const unsigned g = (unsigned)((threads + 255) / 256);
        if (elem_size == 2) pack_row_kernel<__nv_bfloat16><<<g, 256, 0, st>>>(p);
        else pack_row_kernel<float><<<g, 256, 0, st>>>(p);
    }
    return cudaGetLastError();
}

cudaError_t launch_unpack(int elem_size, bool channel_last, const PackParams& p, cudaStream_t st) {
    const int64_t inner = channel_last ? p.dim : p.seqlen;
    const int64_t rows = (int64_t)p.batch * (channel_last ? p.seqlen : p.dim);
    const unsigned g = (unsigned)((rows * ((inner + 7) / 8) + 255) / 256);
#define SSM_UNPACK(T_, CL_)                                                                   \
    if (elem_size == (int)sizeof(T_) && channel_last == CL_) unpack_kernel<T_, CL_><<<g, 256, 0, st>>>(p);
    SSM_UNPACK(__nv_bfloat16, false) SSM_UNPACK(__nv_bfloat16, true)
    SSM_UNPACK(float, false) SSM_UNPACK(float, true)
#undef SSM_UNPACK
    return cudaGetLastError();
}

namespace {
// K<LPR> for rows of NP states a lane
template <int NP, typename F>
void by_lanes(int dstate, F&& f) {
    if (dstate <= NP) f(std::integral_constant<int, 1>{});
    else if (dstate <= 2 * NP) f(std::integral_constant<int, 2>{});
    else if (dstate <= 4 * NP) f(std::integral_constant<int, 4>{});
    else if (dstate <= 8 * NP) f(std::integral_constant<int, 8>{});
    else f(std::integral_constant<int, 16>{});
}
unsigned blocks_of(int64_t threads) { return (unsigned)((threads + 255) / 256); }
}  // namespace

cudaError_t launch_cache_write(const CacheParams& p, cudaStream_t st) {
    by_lanes<8>(p.dstate, [&](auto l) {
        constexpr int L = decltype(l)::value;
        const int64_t per = 256 / L * kCacheRows;
        cache_write_kernel<L><<<(unsigned)((p.batch * p.dim + per - 1) / per), 256, 0, st>>>(p);
    });
    return cudaGetLastError();
}

cudaError_t launch_cache_read(int elem_size, const CacheParams& p, cudaStream_t st) {
    by_lanes<8>(p.dstate, [&](auto l) {
        constexpr int L = decltype(l)::value;
        const unsigned g = blocks_of(p.batch * p.dim * L);
        if (elem_size == 2) cache_read_kernel<__nv_bfloat16, L><<<g, 256, 0, st>>>(p);
        else cache_read_kernel<float, L><<<g, 256, 0, st>>>(p);
    });
    return cudaGetLastError();
}

cudaError_t launch_cached_update(int elem_size, CacheParams p, cudaStream_t st) {
    cudaError_t e = cudaErrorInvalidValue;
    by_lanes<16>(p.dstate, [&](auto l) {
        constexpr int L = decltype(l)::value <= 8 ? decltype(l)::value : 8;
        const int64_t gx = (p.dim + kUpdateThreads / L - 1) / (kUpdateThreads / L);
        // the fewest batch rows a CTA with which all CTAs are resident at once (a second, part
        // wave costs as much as a full one), up to what its shared memory holds
        const int64_t slots = 148 * kUpdateCtas;
        int64_t rows = 1;
        while (rows < update_rows(L) && gx * ((p.batch + rows - 1) / rows) > slots) ++rows;
        p.rows_per_cta = (int)rows;
        // one launch, but for batches of more than 65535 CTAs
        for (int64_t b = 0; b < p.batch; b += 65535ll * p.rows_per_cta) {
            p.first_row = b;
            const int64_t left = (p.batch - b + p.rows_per_cta - 1) / p.rows_per_cta;
            const dim3 g((unsigned)gx, (unsigned)(left < 65535 ? left : 65535));
            auto go = [&](auto elem, auto async, auto heads) {
                cached_update_kernel<decltype(elem), L, decltype(async)::value, decltype(heads)::value>
                    <<<g, kUpdateThreads, 0, st>>>(p);
            };
            auto pick = [&](auto elem) {
                std::true_type yes;
                std::false_type no;
                if (p.async && p.head_dim) go(elem, yes, yes);
                else if (p.async) go(elem, yes, no);
                else if (p.head_dim) go(elem, no, yes);
                else go(elem, no, no);
            };
            if (elem_size == 2) pick(__nv_bfloat16{});
            else pick(float{});
            if ((e = cudaGetLastError()) != cudaSuccess) return;
        }
    });
    return e;
}

}  // namespace ssm

using namespace ssm;

namespace {

// Sizes of an activation that the packing kernels take: their grids hold one thread per 8
// values.
ssm_status_t check_pack(int64_t batch, int64_t dim, int64_t seqlen, ssm_dtype_t dtype) {
    if (bad_dtype(dtype))
        return api_fail(SSM_ERR_BAD_DTYPE, "dtype %d is not SSM_F32 or SSM_BF16", (int)dtype);
    if (batch < 0 || dim < 0 || seqlen < 0) return api_fail(SSM_ERR_BAD_SHAPE, "negative size");
    if (seqlen > 0x3fffffffLL || dim > 0x3fffffffLL)
        return api_fail(SSM_ERR_BAD_SHAPE, "seqlen and dim must be below 2^30");
    if (batch > 65535) return api_fail(SSM_ERR_UNSUPPORTED, "batch %lld > 65535", (long long)batch);
    // one thread per run of 8 along either axis, 256 to a block, below 2^31 blocks
    const double a = (double)batch * dim * (double)(((seqlen + 63) / 64) * 64);
    const double b = (double)batch * seqlen * (double)(((dim + 7) / 8) * 8);
    if (a > 1099511627776.0 || b > 1099511627776.0)
        return api_fail(SSM_ERR_BAD_SHAPE, "batch * dim * seqlen exceeds 2^40");
    return SSM_OK;
}

ssm_status_t check_cache(int64_t batch, int64_t dim, int64_t dstate, int64_t num_slots,
                         const int32_t* slots) {
    if (batch < 0 || dim < 0 || num_slots < 0) return api_fail(SSM_ERR_BAD_SHAPE, "negative size");
    if (dstate < 1 || dstate > SSM_MAX_SCAN_DSTATE)
        return api_fail(SSM_ERR_BAD_SHAPE, "dstate %lld outside 1..%d", (long long)dstate,
                        SSM_MAX_SCAN_DSTATE);
    if (dim > 0x3fffffffLL || batch > 0x3fffffffLL || num_slots > 0x7fffffffLL)
        return api_fail(SSM_ERR_BAD_SHAPE, "batch and dim must be below 2^30, num_slots below 2^31");
    if (batch * dim > 0x7fffffffLL)
        return api_fail(SSM_ERR_BAD_SHAPE, "batch * dim must be below 2^31");
    if (num_slots > 0 && dim > 0xffffffffLL / num_slots)
        return api_fail(SSM_ERR_BAD_SHAPE, "num_slots * dim must be below 2^32");
    if (!slots && num_slots < batch)
        return api_fail(SSM_ERR_BAD_SHAPE, "num_slots %lld < batch %lld without slots",
                        (long long)num_slots, (long long)batch);
    return SSM_OK;
}

}  // namespace

extern "C" {

ssm_status_t ssm_checkpoint_pack(const void* x, void* codes, float* scales, int64_t batch, int64_t dim,
                                 int64_t seqlen, int32_t channel_last, int64_t stride_x,
                                 ssm_dtype_t dtype, ssm_stream_t stream) {
    ssm_status_t status = check_pack(batch, dim, seqlen, dtype);
    if (status != SSM_OK) return status;
    if (channel_last && stride_x != 0 && (stride_x < dim || stride_x > (1ll << 31)))
        return api_fail(SSM_ERR_BAD_SHAPE, "stride_x %lld: 0 or from %lld to 2^31", (long long)stride_x,
                        (long long)dim);
    const int64_t n = batch * dim * seqlen, nb = (seqlen + kBlock8 - 1) / kBlock8;
    if (n == 0) return api_ok();
    if (!x || !codes || !scales)
        return api_fail(SSM_ERR_NULL_ARG, "%s is NULL", !x ? "x" : !codes ? "codes" : "scales");
    const size_t es = size_of(dtype);
    const int64_t sx = channel_last && stride_x ? stride_x : dim;
    const size_t span = channel_last ? (size_t)((batch * seqlen - 1) * sx + dim) * es : (size_t)n * es;
    const Arg ins[] = {{x, es, span, "x"}};
    const Arg outs[] = {{codes, 1, (size_t)n, "codes"}, {scales, 4, (size_t)(batch * dim * nb) * 4, "scales"}};
    if ((status = check_aligned(ins)) != SSM_OK) return status;
    if ((status = check_aligned(outs)) != SSM_OK) return status;
    if ((status = check_alias(outs, ins)) != SSM_OK) return status;
    if ((status = check_distinct(outs)) != SSM_OK) return status;
    PackParams p{x, sx, static_cast<int8_t*>(codes), scales, nullptr, (int)batch, (int)dim, (int)seqlen,
                 is_aligned(x, 16) && sx % 8 == 0};
    cudaError_t e = launch_pack((int)es, channel_last != 0, p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? api_ok() : api_cuda(e, "pack launch");
}

ssm_status_t ssm_checkpoint_unpack(const void* codes, const float* scales, void* out, int64_t batch,
                                   int64_t dim, int64_t seqlen, int32_t channel_last,
                                   ssm_dtype_t dtype, ssm_stream_t stream) {
    ssm_status_t status = check_pack(batch, dim, seqlen, dtype);
    if (status != SSM_OK) return status;
    const int64_t n = batch * dim * seqlen, nb = (seqlen + kBlock8 - 1) / kBlock8;
    if (n == 0) return api_ok();
    if (!codes || !scales || !out)
        return api_fail(SSM_ERR_NULL_ARG, "%s is NULL", !codes ? "codes" : !scales ? "scales" : "out");
    const size_t es = size_of(dtype);
    const Arg ins[] = {{codes, 1, (size_t)n, "codes"}, {scales, 4, (size_t)(batch * dim * nb) * 4, "scales"}};
    const Arg outs[] = {{out, es, (size_t)n * es, "out"}};
    if ((status = check_aligned(ins)) != SSM_OK) return status;
    if ((status = check_aligned(outs)) != SSM_OK) return status;
    if ((status = check_alias(outs, ins)) != SSM_OK) return status;
    PackParams p{nullptr, 0, static_cast<int8_t*>(const_cast<void*>(codes)), const_cast<float*>(scales),
                 out, (int)batch, (int)dim, (int)seqlen, 0};
    cudaError_t e = launch_unpack((int)es, channel_last != 0, p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? api_ok() : api_cuda(e, "unpack launch");
}

ssm_status_t ssm_state_cache_write(const float* state, void* codes, float* scales, const int32_t* slots,
                                   const uint32_t* rand, int64_t batch, int64_t dim, int64_t dstate,
                                   int64_t num_slots, ssm_stream_t stream) {
    ssm_status_t status = check_cache(batch, dim, dstate, num_slots, slots);
    if (status != SSM_OK) return status;
    if (batch * dim == 0 || num_slots == 0) return api_ok();
    if (!state || !codes || !scales)
        return api_fail(SSM_ERR_NULL_ARG, "%s is NULL", !state ? "state" : !codes ? "codes" : "scales");
    const size_t rows = (size_t)batch * dim, held = (size_t)num_slots * dim;
    const Arg ins[] = {{state, 4, rows * dstate * 4, "state"}, {slots, 4, (size_t)batch * 4, "slots"},
                       {rand, 4, rows * 4, "rand"}};
    const Arg outs[] = {{codes, 1, held * dstate, "codes"}, {scales, 4, held * 4, "scales"}};
    if ((status = check_aligned(ins)) != SSM_OK) return status;
    if ((status = check_aligned(outs)) != SSM_OK) return status;
    if ((status = check_alias(outs, ins)) != SSM_OK) return status;
    if ((status = check_distinct(outs)) != SSM_OK) return status;
    CacheParams p{};
    p.batch = batch;
    p.dim = dim;
    p.num_slots = num_slots;
    p.dstate = (int)dstate;
    p.codes = static_cast<int8_t*>(codes);
    p.scales = scales;
    p.slots = slots;
    p.rand = rand;
    p.state = state;
    // every lane of a row holds 8 states of it, at a multiple of 32 bytes
    p.vec = (dstate & (dstate - 1)) == 0 && dstate >= 8 && is_aligned(state, 16);
    cudaError_t e = launch_cache_write(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? api_ok() : api_cuda(e, "cache write launch");
}

ssm_status_t ssm_state_cache_read(const void* codes, const float* scales, const int32_t* slots, void* out,
                                  int64_t batch, int64_t dim, int64_t dstate, int64_t num_slots,
                                  ssm_dtype_t dtype, ssm_stream_t stream) {
    if (bad_dtype(dtype))
        return api_fail(SSM_ERR_BAD_DTYPE, "dtype %d is not SSM_F32 or SSM_BF16", (int)dtype);
    ssm_status_t status = check_cache(batch, dim, dstate, num_slots, slots);
    if (status != SSM_OK) return status;
    if (batch * dim == 0 || num_slots == 0) return api_ok();
    if (!codes || !scales || !out)
        return api_fail(SSM_ERR_NULL_ARG, "%s is NULL", !codes ? "codes" : !scales ? "scales" : "out");
    const size_t es = size_of(dtype), rows = (size_t)batch * dim, held = (size_t)num_slots * dim;
    const Arg ins[] = {{codes, 1, held * dstate, "codes"}, {scales, 4, held * 4, "scales"},
                       {slots, 4, (size_t)batch * 4, "slots"}};
    const Arg outs[] = {{out, es, rows * dstate * es, "out"}};
    if ((status = check_aligned(ins)) != SSM_OK) return status;
    if ((status = check_aligned(outs)) != SSM_OK) return status;
    if ((status = check_alias(outs, ins)) != SSM_OK) return status;
    CacheParams p{};
    p.batch = batch;
    p.dim = dim;
    p.num_slots = num_slots;
    p.dstate = (int)dstate;
    p.codes = static_cast<int8_t*>(const_cast<void*>(codes));
    p.scales = const_cast<float*>(scales);
    p.slots = slots;
    p.out = out;
    cudaError_t e = launch_cache_read((int)es, p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? api_ok() : api_cuda(e, "cache read launch");
}

ssm_status_t ssm_selective_state_update_cached(const ssm_cached_update_args_t* a, ssm_stream_t stream) {
    if (!a) return api_fail(SSM_ERR_NULL_ARG, "args is NULL");
    if (bad_dtype(a->dtype))
        return api_fail(SSM_ERR_BAD_DTYPE, "dtype %d is not SSM_F32 or SSM_BF16", (int)a->dtype);
    ssm_status_t status = check_cache(a->batch, a->dim, a->dstate, a->num_slots, a->slots);
    if (status != SSM_OK) return status;
    if (a->a_heads < 0 || (a->a_heads > 0 && a->dim % a->a_heads != 0))
        return api_fail(SSM_ERR_BAD_SHAPE, "a_heads %d must be 0 or divide dim %lld", a->a_heads,
                        (long long)a->dim);
    if (a->conv_weight && (a->conv_width < 1 || a->conv_width > SSM_MAX_CONV_WIDTH))
        return api_fail(SSM_ERR_BAD_SHAPE, "conv_width %d outside 1..%d", a->conv_width,
                        SSM_MAX_CONV_WIDTH);
    if (a->batch * a->dim == 0 || a->num_slots == 0) return api_ok();
    struct { const void* p; const char* n; } req[] = {
        {a->codes, "codes"}, {a->scales, "scales"}, {a->x, "x"}, {a->dt, "dt"}, {a->A, "A"},
        {a->B_t, "B_t"}, {a->C_t, "C_t"}, {a->out, "out"}};
    for (auto& r : req)
        if (!r.p) return api_fail(SSM_ERR_NULL_ARG, "%s is NULL", r.n);
    if (a->conv_weight && !a->conv_state) return api_fail(SSM_ERR_NULL_ARG, "conv_state is NULL");
    const size_t es = size_of(a->dtype), rows = (size_t)a->batch * a->dim;
    const size_t held = (size_t)a->num_slots * a->dim, D = (size_t)a->dim;
    const size_t bc = (size_t)a->batch * a->dstate * es, wb = a->conv_weight ? D * a->conv_width * 4 : 0;
    const Arg ins[] = {
        {a->x, es, rows * es, "x"}, {a->dt, es, rows * es, "dt"}, {a->z, es, rows * es, "z"},
        {a->B_t, es, bc, "B_t"}, {a->C_t, es, bc, "C_t"},
        {a->A, 4, (a->a_heads > 0 ? (size_t)a->a_heads : D * a->dstate) * 4, "A"},
        {a->D, 4, D * 4, "D"}, {a->dt_bias, 4, D * 4, "dt_bias"}, {a->conv_weight, 4, wb, "conv_weight"},
        {a->conv_bias, 4, D * 4, "conv_bias"}, {a->slots, 4, (size_t)a->batch * 4, "slots"},
        {a->rand, 4, rows * 4, "rand"}};
    const Arg outs[] = {{a->codes, 1, held * a->dstate, "codes"}, {a->scales, 4, held * 4, "scales"},
                        {a->conv_weight ? a->conv_state : nullptr, es,
                         a->conv_weight ? held * a->conv_width * es : 0, "conv_state"},
                        {a->out, es, rows * es, "out"}};
    if ((status = check_aligned(ins)) != SSM_OK) return status;
    if ((status = check_aligned(outs)) != SSM_OK) return status;
    if ((status = check_alias(outs, ins)) != SSM_OK) return status;
    if ((status = check_distinct(outs)) != SSM_OK) return status;
    CacheParams p{};
    p.batch = a->batch;
    p.dim = a->dim;
    p.num_slots = a->num_slots;
    p.dstate = (int)a->dstate;
    p.codes = static_cast<int8_t*>(a->codes);
    p.scales = a->scales;
    p.slots = a->slots;
    p.rand = a->rand;
    p.out = a->out;
    p.conv_state = a->conv_weight ? a->conv_state : nullptr;
    p.x = a->x;
    p.dt = a->dt;
    p.Bt = a->B_t;
    p.Ct = a->C_t;
    p.z = a->z;
    p.A = a->A;
    p.D = a->D;
    p.dt_bias = a->dt_bias;
    p.conv_w = a->conv_weight;
    p.conv_b = a->conv_weight ? a->conv_bias : nullptr;
    p.conv_width = a->conv_weight ? a->conv_width : 0;
    p.softplus = a->dt_softplus ? 1 : 0;
    p.head_dim = a->a_heads > 0 ? (int)(a->dim / a->a_heads) : 0;
    p.async = a->dstate % 16 == 0 && is_aligned(a->codes, 16) &&
              (!a->conv_weight || (a->conv_width == 4 && is_aligned(a->conv_state, 4 * es)));
    cudaError_t e = launch_cached_update((int)es, p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? api_ok() : api_cuda(e, "cached state update launch");
}

}  // extern "C"
