// rq_tmix_api.cu -- argument checks of the time-mix recurrence's calls.
#include "rq_tmix.cuh"

using namespace rq;

namespace {

bool mis(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

rq_status failed(cudaError_t e) {
    if (e == cudaSuccess) return RQ_OK;
    record_cuda_error(e);
    return RQ_ERR_CUDA;
}

// T tokens of H heads in S sequences.
rq_status check_sizes(int64_t T, int64_t H, int64_t S, int64_t ld, int dtype) {
    if (dtype != RQ_OUT_F32 && dtype != RQ_OUT_F16) return RQ_ERR_RANGE;
    if (T < 0 || T >= (int64_t{1} << 30) || H < 1 || H > (1 << 20) || S < 1 || S >= (1 << 30)) return RQ_ERR_SHAPE;
    if (ld < H * kHead || ld % 8 != 0 || ld >= (int64_t{1} << 40)) return RQ_ERR_SHAPE;
    if ((T / kTmixChunk + S) * H * 4 >= (int64_t{1} << 31)) return RQ_ERR_SHAPE;   // blocks of a launch
    return RQ_OK;
}

rq_status check_tokens(const void* const* p, int n, int64_t T) {
    for (int i = 0; i < n; ++i)
        if (p[i] == nullptr && T > 0) return RQ_ERR_NULL;
    for (int i = 0; i < n; ++i)
        if (mis(p[i], 16)) return RQ_ERR_ALIGN;
    return RQ_OK;
}

}  // namespace

extern "C" {

size_t rq_tmix_ckpt_bytes(int64_t T, int64_t S, int64_t H) {
    if (check_sizes(T, H, S, H * kHead, RQ_OUT_F32) != RQ_OK) return 0;
    return static_cast<size_t>(T / kTmixChunk + S) * H * kHead * kHead * sizeof(float);
}

rq_status rq_tmix_scan(const void* r, const void* d, const void* k, const void* v, const void* a, const void* b,
                       int64_t T, int64_t H, int64_t ld, int dtype, const int32_t* seq_start, int64_t S,
                       const float* state_in, float* state_out, const int32_t* slots, int64_t n_slots, void* y,
                       float* ckpt, int* dev_status, rq_stream_t stream) {
    rq_status st = check_sizes(T, H, S, ld, dtype);
    if (st != RQ_OK) return st;
    if (slots != nullptr && n_slots < 1) return RQ_ERR_SHAPE;
    if (seq_start == nullptr) return RQ_ERR_NULL;
    const void* tokens[7] = {r, d, k, v, a, b, y};
    if ((st = check_tokens(tokens, 7, T)) != RQ_OK) return st;
    if (mis(state_in, 16) || mis(state_out, 16) || mis(ckpt, 16) || mis(seq_start, 4) || mis(slots, 4) ||
        mis(dev_status, 4))
        return RQ_ERR_ALIGN;
    TmixArgs p = {};
    for (int i = 0; i < 6; ++i) p.in[i] = tokens[i];
    p.out[0] = y;
    p.state_in = state_in;
    p.state_out = state_out;
    p.slots = slots;
    p.n_slots = n_slots;
    p.seq_start = seq_start;
    p.ckpt = ckpt;
    p.status = dev_status;
    p.T = T;
    p.ld = ld;
    p.S = static_cast<int>(S);
    p.H = static_cast<int>(H);
    return failed(launch_tmix_scan(p, dtype == RQ_OUT_F16, false, reinterpret_cast<cudaStream_t>(stream)));
}

rq_status rq_tmix_scan_bwd(const void* r, const void* d, const void* k, const void* v, const void* a,
                           const void* b, int64_t T, int64_t H, int64_t ld, int dtype, const int32_t* seq_start,
                           int64_t S, const float* ckpt, const void* dy, const float* dstate_out, float* dstate_in,
                           void* dr, void* dd, void* dk, void* dv, void* da, void* db, float* work,
                           int* dev_status, rq_stream_t stream) {
    rq_status st = check_sizes(T, H, S, ld, dtype);
    if (st != RQ_OK) return st;
    if (seq_start == nullptr || ckpt == nullptr || work == nullptr) return RQ_ERR_NULL;
    const void* tokens[13] = {r, d, k, v, a, b, dy, dr, dd, dk, dv, da, db};
    if ((st = check_tokens(tokens, 13, T)) != RQ_OK) return st;
    if (mis(dstate_in, 16) || mis(dstate_out, 16) || mis(ckpt, 16) || mis(work, 16) || mis(seq_start, 4) ||
        mis(dev_status, 4))
        return RQ_ERR_ALIGN;
    TmixArgs p = {};
    for (int i = 0; i < 6; ++i) p.in[i] = tokens[i];
    p.dy = dy;
    void* grads[6] = {dr, dd, dk, dv, da, db};
    for (int i = 0; i < 6; ++i) p.out[i] = grads[i];
    p.state_in = dstate_out;                 // the walk runs from the last token to the first
    p.state_out = dstate_in;
    p.seq_start = seq_start;
    p.ckpt = const_cast<float*>(ckpt);
    p.gckpt = work;
    p.status = dev_status;
    p.T = T;
    p.ld = ld;
    p.S = static_cast<int>(S);
    p.H = static_cast<int>(H);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = launch_tmix_scan(p, dtype == RQ_OUT_F16, true, s);
    if (e == cudaSuccess && T > 0) e = launch_tmix_chunks_bwd(p, dtype == RQ_OUT_F16, s);
    return failed(e);
}

rq_status rq_tmix_step(const void* r, const void* d, const void* k, const void* v, const void* a, const void* b,
                       int64_t B, int64_t H, int64_t ld, int dtype, const float* state_in, float* state_out,
                       const int32_t* slots, int64_t n_slots, void* y, int* dev_status, rq_stream_t stream) {
    if (B < 1) return RQ_ERR_SHAPE;
    rq_status st = check_sizes(B, H, B, ld, dtype);
    if (st != RQ_OK) return st;
    if (slots != nullptr && n_slots < 1) return RQ_ERR_SHAPE;
    const void* tokens[7] = {r, d, k, v, a, b, y};
    if ((st = check_tokens(tokens, 7, B)) != RQ_OK) return st;
    if (mis(state_in, 16) || mis(state_out, 16) || mis(slots, 4) || mis(dev_status, 4)) return RQ_ERR_ALIGN;
    TmixArgs p = {};
    for (int i = 0; i < 6; ++i) p.in[i] = tokens[i];
    p.out[0] = y;
    p.state_in = state_in;
    p.state_out = state_out;
    p.slots = slots;
    p.n_slots = n_slots;
    p.status = dev_status;
    p.T = B;
    p.ld = ld;
    p.S = static_cast<int>(B);
    p.H = static_cast<int>(H);
    return failed(launch_tmix_step(p, dtype == RQ_OUT_F16, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
