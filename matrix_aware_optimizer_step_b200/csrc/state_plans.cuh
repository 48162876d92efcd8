// state_plans.cuh -- host side of the plans over lists of tensors (AdamW with
// 32- or 8-bit moments, gradient norm, moment conversion).  Included by
// muon_abi.cu after its helpers.
//
// A plan lays its tensors out once, as a device table of chunks, so that a
// call is argument checks and launches: nothing is copied to the device, no
// memory is allocated, and the call can be captured into a CUDA graph.  The
// table never changes after creation.  Gradients, which a training loop may
// reallocate every step, are the exception: their pointers stay on the host
// and travel as a kernel parameter.
#pragma once

#include <new>

namespace {
enum PlanKind { PLAN_ADAMW, PLAN_NORM, PLAN_STATE8 };
}  // namespace

// One launch: up to MAX_SLOTS tensors of one combination of types.
struct PlanBucket {
  int pbf16 = 0, gbf16 = 0, copy = 0;
  std::vector<int> tensors;      // places in the plan's list; index = slot
  size_t first = 0, chunks = 0;  // in the plan's table
  int blocks = 1;                // of 256 elements, per warp (AdamW)
};

struct muon_plan {
  muon_ctx* ctx = nullptr;       // nullptr once the context was destroyed
  PlanKind kind = PLAN_ADAMW;
  int device = 0;
  int state_bits = 32;
  void* table = nullptr;
  std::vector<const void*> grads;
  std::vector<int64_t> grad_numel;
  std::vector<int> grad_size;        // bytes of one element
  std::vector<std::pair<uintptr_t, uintptr_t>> written;   // sorted, disjoint
  std::vector<PlanBucket> buckets;
  std::vector<unsigned> norm_grid;
  unsigned norm_ctas = 0;        // of all launches
};

namespace {

// The caller's current device is put back when a call returns.
struct DeviceGuard {
  int prev = -1;
  cudaError_t err;
  explicit DeviceGuard(int device) {
    err = cudaGetDevice(&prev);
    if (err == cudaSuccess && prev != device) err = cudaSetDevice(device);
    else if (err == cudaSuccess) prev = -1;
  }
  ~DeviceGuard() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

constexpr int64_t kMaxNumel = int64_t(1) << 38;   // no GPU holds more

// Plans may be freed by a garbage collector's thread.
std::mutex g_plans_mutex;

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Span {
  uintptr_t lo, hi;
  bool writes;
};

// Whether anything written overlaps anything else; `spans` comes back sorted.
bool overlapping(std::vector<Span>& spans) {
  std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
  uintptr_t any = 0, wrote = 0;
  for (const Span& s : spans) {
    if (s.lo < (s.writes ? any : wrote)) return true;
    any = std::max(any, s.hi);
    if (s.writes) wrote = std::max(wrote, s.hi);
  }
  return false;
}

void add_span(std::vector<Span>& v, const void* p, int64_t bytes, bool writes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  if (p && bytes > 0) v.push_back({a, a + uintptr_t(bytes), writes});
}

int dtype_size(int dt) { return dt == MUON_BF16 ? 2 : 4; }

constexpr size_t kMaxChunks = (size_t(1) << 31) - 1;   // blocks of one launch

// Upload the table and register the plan with its context.
template <typename T>
muon_status finish_plan(muon_ctx* ctx, muon_plan* plan, const std::vector<T>& table, muon_plan** out) {
  for (const PlanBucket& b : plan->buckets)
    if (b.chunks > kMaxChunks) return fail(ctx, MUON_ERR_UNSUPPORTED, "more elements than one launch covers");
  if (!table.empty()) {
    CUDA_TRY(ctx, cudaMalloc(&plan->table, table.size() * sizeof(T)));
    cudaError_t e = cudaMemcpyAsync(plan->table, table.data(), table.size() * sizeof(T), cudaMemcpyHostToDevice,
                                    cudaStreamPerThread);
    if (e == cudaSuccess) e = cudaStreamSynchronize(cudaStreamPerThread);
    if (e != cudaSuccess) {
      cudaFree(plan->table);
      plan->table = nullptr;
      return fail(ctx, MUON_ERR_CUDA, "table upload failed: %s", cudaGetErrorString(e));
    }
  }
  std::lock_guard<std::mutex> lock(g_plans_mutex);
  ctx->plans.push_back(plan);
  *out = plan;
  return MUON_OK;
}

// Run `body(plan)` on a new plan; every failure frees it.
template <typename F>
muon_status make_plan(muon_ctx* ctx, muon_plan** out, PlanKind kind, F&& body) {
  if (!ctx || !out) return MUON_ERR_INVALID_ARG;
  *out = nullptr;
  muon_plan* plan = nullptr;
  muon_status s;
  try {
    DeviceGuard guard(ctx->device);
    CUDA_TRY(ctx, guard.err);
    CUDA_TRY(ctx, cudaGetLastError());
    plan = new muon_plan();
    plan->ctx = ctx;
    plan->kind = kind;
    plan->device = ctx->device;
    s = body(plan);
  } catch (const std::exception&) {
    s = fail(ctx, MUON_ERR_WORKSPACE, "out of host memory");
  }
  if (s != MUON_OK) {
    *out = nullptr;
    if (plan && plan->table) cudaFree(plan->table);
    delete plan;
  }
  return s;
}

muon_status check_plan(muon_plan* plan, PlanKind kind) {
  if (!plan || !plan->ctx) return MUON_ERR_INVALID_ARG;
  if (plan->kind != kind) return fail(plan->ctx, MUON_ERR_INVALID_ARG, "the plan is of another kind");
  return MUON_OK;
}

void fill_grads(const muon_plan* plan, const PlanBucket& b, GradPtrs& g) {
  for (size_t k = 0; k < b.tensors.size(); ++k) g.p[k] = plan->grads[b.tensors[k]];
}

// Tensors of one key in list order, MAX_SLOTS per bucket.
PlanBucket& bucket_for(muon_plan* plan, int pbf16, int gbf16, int copy) {
  for (size_t k = plan->buckets.size(); k-- > 0;) {
    PlanBucket& b = plan->buckets[k];
    if (b.pbf16 == pbf16 && b.gbf16 == gbf16 && b.copy == copy) {
      if (b.tensors.size() < size_t(MAX_SLOTS)) return b;
      break;
    }
  }
  plan->buckets.emplace_back();
  plan->buckets.back().pbf16 = pbf16;
  plan->buckets.back().gbf16 = gbf16;
  plan->buckets.back().copy = copy;
  return plan->buckets.back();
}

// Load a kernel on the current device ahead of its first launch, which may
// happen inside a stream capture, where nothing should be loaded.
template <typename... KArgs>
cudaError_t load_kernel(void (*kernel)(KArgs...)) {
  cudaFuncAttributes a;
  return cudaFuncGetAttributes(&a, kernel);
}

// load: make the kernel ready instead of launching it.
template <bool S8, bool P, bool C, bool G, bool ST>
cudaError_t launch_adamw(const muon_plan* plan, const PlanBucket& b, const GradPtrs& g, const AdamPlanScalars& sc,
                         int* flags, cudaStream_t st, bool load) {
  const AdamChunk* t = static_cast<const AdamChunk*>(plan->table) + b.first;
  const dim3 grid{unsigned(b.chunks)};
  if constexpr (S8) {
    constexpr int smem = Stage8<P, G>::cta;
    if (load)
      return cudaFuncSetAttribute(adamw8_kernel<P, C, G, ST>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    return launch_pdl(adamw8_kernel<P, C, G, ST>, grid, dim3(ST_THREADS), size_t(smem), st, t, b.blocks, g, sc, flags);
  } else {
    if (load) return load_kernel(adamw32_kernel<P, C, G, ST>);
    return launch_pdl(adamw32_kernel<P, C, G, ST>, grid, dim3(ST_THREADS), size_t(0), st, t, g, sc,
                      static_cast<const int*>(flags));
  }
}

using AdamLaunch = cudaError_t (*)(const muon_plan*, const PlanBucket&, const GradPtrs&, const AdamPlanScalars&, int*,
                                   cudaStream_t, bool);

// A copy goes with fp32 parameters only.  Stochastic rounding concerns codes
// and bf16 parameters: fp32 moments on fp32 parameters have nothing to round.
template <bool S8, bool P, bool C>
AdamLaunch pick_adamw(bool g, bool stoch) {
  if (stoch && (S8 || P)) return g ? launch_adamw<S8, P, C, true, S8 || P> : launch_adamw<S8, P, C, false, S8 || P>;
  return g ? launch_adamw<S8, P, C, true, false> : launch_adamw<S8, P, C, false, false>;
}

AdamLaunch adamw_launcher(bool s8, const PlanBucket& b, bool stoch) {
  if (s8)
    return b.pbf16 ? pick_adamw<true, true, false>(b.gbf16, stoch)
                   : b.copy ? pick_adamw<true, false, true>(b.gbf16, stoch) : pick_adamw<true, false, false>(b.gbf16, stoch);
  return b.pbf16 ? pick_adamw<false, true, false>(b.gbf16, stoch)
                 : b.copy ? pick_adamw<false, false, true>(b.gbf16, stoch) : pick_adamw<false, false, false>(b.gbf16, stoch);
}

}  // namespace

extern "C" {

void muon_default_adamw_plan_hparams(muon_adamw_plan_hparams* hp) {
  if (!hp) return;
  hp->lr = 3e-4;
  hp->beta1 = 0.9;
  hp->beta2 = 0.95;
  hp->eps = 1e-8;
  hp->weight_decay = 0.01;
}

muon_status muon_adamw_plan_create(muon_ctx* ctx, const muon_plan_tensor* tensors, int32_t n, int32_t state_bits,
                                   muon_plan** out) {
  return make_plan(ctx, out, PLAN_ADAMW, [&](muon_plan* plan) -> muon_status {
    if (n < 0 || (n > 0 && !tensors)) return fail(ctx, MUON_ERR_INVALID_ARG, "bad tensor list");
    if (state_bits != 8 && state_bits != 32)
      return fail(ctx, MUON_ERR_INVALID_ARG, "state_bits %d: 8 or 32", state_bits);
    const bool s8 = state_bits == 8;
    plan->state_bits = state_bits;
    std::vector<Span> spans;
    for (int i = 0; i < n; ++i) {
      const muon_plan_tensor& t = tensors[i];
      if (t.numel < 0 || t.numel > kMaxNumel)
        return fail(ctx, MUON_ERR_INVALID_ARG, "tensor %d: numel %lld", i, (long long)t.numel);
      if ((t.param_dtype != MUON_F32 && t.param_dtype != MUON_BF16) ||
          (t.grad_dtype != MUON_F32 && t.grad_dtype != MUON_BF16))
        return fail(ctx, MUON_ERR_INVALID_ARG, "tensor %d: param_dtype %d, grad_dtype %d", i, t.param_dtype,
                    t.grad_dtype);
      plan->grads.push_back(t.grad);
      plan->grad_numel.push_back(t.numel);
      plan->grad_size.push_back(dtype_size(t.grad_dtype));
      if (t.numel == 0) continue;
      if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq || (s8 && (!t.exp_avg_scale || !t.exp_avg_sq_scale)))
        return fail(ctx, MUON_ERR_INVALID_ARG, "tensor %d: NULL pointer", i);
      if (!s8 && (t.exp_avg_scale || t.exp_avg_sq_scale))
        return fail(ctx, MUON_ERR_INVALID_ARG, "tensor %d: scales belong to 8-bit moments", i);
      if (t.param_copy && t.param_dtype != MUON_F32)
        return fail(ctx, MUON_ERR_INVALID_ARG, "tensor %d: a bf16 copy goes with an fp32 parameter", i);
      if (!aligned_to(t.param, dtype_size(t.param_dtype)) || !aligned_to(t.grad, dtype_size(t.grad_dtype)) ||
          !aligned_to(t.param_copy, 2) || !aligned_to(t.exp_avg_scale, 4) || !aligned_to(t.exp_avg_sq_scale, 4) ||
          (!s8 && (!aligned_to(t.exp_avg, 4) || !aligned_to(t.exp_avg_sq, 4))))
        return fail(ctx, MUON_ERR_INVALID_ARG, "tensor %d: a pointer is not aligned to its element", i);
      const int64_t blocks = cdiv(t.numel, Q_BLOCK);
      add_span(spans, t.param, t.numel * dtype_size(t.param_dtype), true);
      add_span(spans, t.param_copy, t.numel * 2, true);
      add_span(spans, t.exp_avg, t.numel * (s8 ? 1 : 4), true);
      add_span(spans, t.exp_avg_sq, t.numel * (s8 ? 1 : 4), true);
      add_span(spans, t.exp_avg_scale, blocks * 4, true);
      add_span(spans, t.exp_avg_sq_scale, blocks * 4, true);
      add_span(spans, t.grad, t.numel * dtype_size(t.grad_dtype), false);
      bucket_for(plan, t.param_dtype == MUON_BF16, t.grad_dtype == MUON_BF16, t.param_copy != nullptr).tensors.push_back(i);
    }
    if (overlapping(spans))
      return fail(ctx, MUON_ERR_INVALID_ARG, "a tensor that the step writes overlaps another tensor of the plan");
    for (const Span& s : spans)
      if (s.writes) plan->written.push_back({s.lo, s.hi});
    // 8-bit: as many blocks per warp as give the resident warps one turn, up
    // to what their shared memory holds; few blocks are spread over more warps
    int64_t total = 0;
    for (int i = 0; i < n; ++i) total += cdiv(tensors[i].numel, int64_t(Q_BLOCK));
    const int64_t turn = total / (int64_t(device_sms(ctx->device)) * ADAM8_CTAS * ST_WARPS);
    std::vector<AdamChunk> table;
    for (PlanBucket& b : plan->buckets) {
      b.first = table.size();
      const int most = b.pbf16 ? (b.gbf16 ? Stage8<true, true>::blocks : Stage8<true, false>::blocks)
                               : (b.gbf16 ? Stage8<false, true>::blocks : Stage8<false, false>::blocks);
      b.blocks = s8 ? int(std::min<int64_t>(std::max<int64_t>(turn, 1), most)) : 1;
      const int64_t chunk = int64_t(b.blocks) * ST_WARPS * Q_BLOCK;
      size_t more = 0;
      for (int i : b.tensors) more += size_t(cdiv(tensors[i].numel, chunk));
      table.reserve(table.size() + more);
      for (size_t k = 0; k < b.tensors.size(); ++k) {
        const muon_plan_tensor& t = tensors[b.tensors[k]];
        const int64_t es = s8 ? 1 : 4;
        for (int64_t at = 0; at < t.numel; at += chunk) {
          AdamChunk c{};
          c.param = static_cast<char*>(t.param) + at * dtype_size(t.param_dtype);
          c.m = static_cast<char*>(t.exp_avg) + at * es;
          c.v = static_cast<char*>(t.exp_avg_sq) + at * es;
          c.m_scale = s8 ? t.exp_avg_scale + at / Q_BLOCK : nullptr;
          c.v_scale = s8 ? t.exp_avg_sq_scale + at / Q_BLOCK : nullptr;
          c.copy = t.param_copy ? static_cast<__nv_bfloat16*>(t.param_copy) + at : nullptr;
          c.base = at;
          c.id = uint32_t(b.tensors[k]);
          c.slot = uint16_t(k);
          c.count = uint16_t(std::min<int64_t>(chunk, t.numel - at));
          table.push_back(c);
        }
      }
      b.chunks = table.size() - b.first;
      for (int stochastic = 0; stochastic < 2; ++stochastic)
        CUDA_TRY(ctx, adamw_launcher(s8, b, stochastic != 0)(plan, b, GradPtrs{}, AdamPlanScalars{}, nullptr, nullptr, true));
    }
    return finish_plan(ctx, plan, table, out);
  });
}

muon_status muon_adamw_plan_step(muon_plan* plan, const muon_adamw_plan_hparams* hp, int64_t step,
                                 const int64_t* step_ptr, const float* lr_ptr, const float* grad_scale,
                                 int32_t stochastic, uint32_t seed, void* stream) {
  muon_status s = check_plan(plan, PLAN_ADAMW);
  if (s != MUON_OK) return s;
  muon_ctx* ctx = plan->ctx;
  if (!hp) return fail(ctx, MUON_ERR_INVALID_ARG, "hparams is NULL");
  if (!step_ptr && step < 1) return fail(ctx, MUON_ERR_INVALID_ARG, "step counts from 1");
  if (!(hp->beta1 >= 0. && hp->beta1 < 1. && hp->beta2 >= 0. && hp->beta2 < 1. && float(hp->eps) > 0.f))
    return fail(ctx, MUON_ERR_INVALID_ARG, "betas must lie in [0,1), eps > 0");
  if (!std::isfinite(float(hp->lr)) || !std::isfinite(float(hp->weight_decay)) || !std::isfinite(float(hp->eps)))
    return fail(ctx, MUON_ERR_INVALID_ARG, "non-finite hyper-parameter");
  if (!aligned_to(step_ptr, 8) || !aligned_to(lr_ptr, 4) || !aligned_to(grad_scale, 4))
    return fail(ctx, MUON_ERR_INVALID_ARG, "a device scalar is not aligned to its type");
  for (const PlanBucket& b : plan->buckets)
    for (int i : b.tensors)
      if (!plan->grads[i]) return fail(ctx, MUON_ERR_INVALID_ARG, "tensor %d: NULL gradient", i);
  if (plan->buckets.empty()) return MUON_OK;
  DeviceGuard guard(plan->device);
  CUDA_TRY(ctx, guard.err);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  ctx->last_stream = st;
  CUDA_TRY(ctx, cudaGetLastError());
  AdamPlanScalars sc{};
  auto twice = [](double x) { return make_float2(float(x), float(x)); };
  sc.beta1 = twice(hp->beta1);
  sc.one_beta1 = twice(1.0 - hp->beta1);
  sc.beta2 = twice(hp->beta2);
  sc.one_beta2 = twice(1.0 - hp->beta2);
  sc.eps = float(hp->eps);
  sc.eps2 = twice(hp->eps);
  sc.minus_zero = twice(-0.0);
  sc.decay = float(1.0 - hp->lr * hp->weight_decay);
  sc.lr = hp->lr;
  sc.wd = hp->weight_decay;
  sc.ln_beta1 = std::log(hp->beta1);
  sc.ln_beta2 = std::log(hp->beta2);
  if (!step_ptr) {
    const double bc1 = -std::expm1(double(step) * sc.ln_beta1), bc2 = -std::expm1(double(step) * sc.ln_beta2);
    sc.step_size = float((lr_ptr ? 1.0 : hp->lr) / bc1);   // the kernel multiplies a device rate in
    sc.inv_bc2 = float(1.0 / std::sqrt(bc2));
    sc.step = uint32_t(uint64_t(step));
  }
  sc.step_ptr = step_ptr;
  sc.lr_ptr = lr_ptr;
  sc.grad_scale = grad_scale;
  sc.seed_key = mix32(seed);
  GradPtrs g;
  ProfScope ps(ctx, MUON_K_ADAMW, st);
  for (const PlanBucket& b : plan->buckets) {
    fill_grads(plan, b, g);
    const AdamLaunch f = adamw_launcher(plan->state_bits == 8, b, stochastic != 0);
    CUDA_TRY(ctx, f(plan, b, g, sc, ctx->dflags, st, false));
    ctx->launches++;
  }
  return MUON_OK;
}

muon_status muon_grad_norm_plan_create(muon_ctx* ctx, const muon_grad_tensor* tensors, int32_t n, muon_plan** out) {
  return make_plan(ctx, out, PLAN_NORM, [&](muon_plan* plan) -> muon_status {
    if (n < 0 || (n > 0 && !tensors)) return fail(ctx, MUON_ERR_INVALID_ARG, "bad tensor list");
    for (int i = 0; i < n; ++i) {
      const muon_grad_tensor& t = tensors[i];
      if (t.numel < 0 || t.numel > kMaxNumel)
        return fail(ctx, MUON_ERR_INVALID_ARG, "tensor %d: numel %lld", i, (long long)t.numel);
      if (t.grad_dtype != MUON_F32 && t.grad_dtype != MUON_BF16)
        return fail(ctx, MUON_ERR_INVALID_ARG, "tensor %d: grad_dtype %d", i, t.grad_dtype);
      plan->grads.push_back(t.grad);
      plan->grad_numel.push_back(t.numel);
      plan->grad_size.push_back(dtype_size(t.grad_dtype));
      if (t.numel == 0) continue;
      if (!t.grad) return fail(ctx, MUON_ERR_INVALID_ARG, "tensor %d: NULL pointer", i);
      if (!aligned_to(t.grad, dtype_size(t.grad_dtype)))
        return fail(ctx, MUON_ERR_INVALID_ARG, "tensor %d: a pointer is not aligned to its element", i);
      bucket_for(plan, 0, 0, 0).tensors.push_back(i);
    }
    std::vector<NormChunk> table;
    const size_t most = size_t(device_sms(ctx->device)) * NORM_CTAS;
    for (PlanBucket& b : plan->buckets) {
      b.first = table.size();
      for (size_t k = 0; k < b.tensors.size(); ++k) {
        const muon_grad_tensor& t = tensors[b.tensors[k]];
        const int64_t chunk = NORM_BYTES / dtype_size(t.grad_dtype);
        for (int64_t at = 0; at < t.numel; at += chunk)
          table.push_back({at, uint16_t(k), uint16_t(std::min(chunk, t.numel - at)), t.grad_dtype == MUON_BF16 ? 1u : 0u});
      }
      b.chunks = table.size() - b.first;
      plan->norm_grid.push_back(unsigned(std::min(b.chunks, most)));
      plan->norm_ctas += plan->norm_grid.back();
    }
    CUDA_TRY(ctx, load_kernel(grad_norm_kernel));
    return finish_plan(ctx, plan, table, out);
  });
}

muon_status muon_grad_norm_out_bytes(const muon_plan* plan, size_t* bytes) {
  if (!plan || !bytes || plan->kind != PLAN_NORM) return MUON_ERR_INVALID_ARG;
  *bytes = 16 + size_t(plan->norm_ctas) * sizeof(double);
  return MUON_OK;
}

muon_status muon_grad_norm_run(muon_plan* plan, double max_norm, float* out, void* stream) {
  muon_status s = check_plan(plan, PLAN_NORM);
  if (s != MUON_OK) return s;
  muon_ctx* ctx = plan->ctx;
  if (!out || !aligned_to(out, 16)) return fail(ctx, MUON_ERR_INVALID_ARG, "out is NULL or not 16-byte aligned");
  if (!(max_norm >= 0.0)) return fail(ctx, MUON_ERR_INVALID_ARG, "max_norm must be >= 0");
  for (const PlanBucket& b : plan->buckets)
    for (int i : b.tensors)
      if (!plan->grads[i]) return fail(ctx, MUON_ERR_INVALID_ARG, "tensor %d: NULL gradient", i);
  DeviceGuard guard(plan->device);
  CUDA_TRY(ctx, guard.err);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  ctx->last_stream = st;
  CUDA_TRY(ctx, cudaGetLastError());
  NormOut o{};
  o.out = out;
  o.counter = reinterpret_cast<unsigned int*>(out + 2);
  o.partials = reinterpret_cast<double*>(out + 4);
  o.max_norm = max_norm;
  o.total = plan->norm_ctas;
  GradPtrs g;
  ProfScope ps(ctx, MUON_K_OTHER, st);
  for (size_t k = 0; k < plan->buckets.size(); ++k) {
    const PlanBucket& b = plan->buckets[k];
    fill_grads(plan, b, g);
    const cudaError_t e = launch_pdl(grad_norm_kernel, dim3(plan->norm_grid[k]), dim3(ST_THREADS), size_t(0), st,
                                     static_cast<const NormChunk*>(plan->table) + b.first, unsigned(b.chunks), g, o);
    if (e != cudaSuccess) {      // launches that did go out must not leave a count for the next run
      cudaMemsetAsync(o.counter, 0, sizeof(unsigned int), st);
      return fail(ctx, MUON_ERR_CUDA, "grad_norm launch failed: %s", cudaGetErrorString(e));
    }
    ctx->launches++;
    o.first += plan->norm_grid[k];
  }
  if (plan->buckets.empty()) {     // nothing to sum: norm 0
    CUDA_TRY(ctx, launch_pdl(grad_norm_kernel, dim3(1), dim3(ST_THREADS), size_t(0), st,
                             static_cast<const NormChunk*>(nullptr), 0u, g, o));
    ctx->launches++;
  }
  return MUON_OK;
}

muon_status muon_plan_bind_grads(muon_plan* plan, const void* const* grads, int32_t n) {
  if (!plan || !plan->ctx) return MUON_ERR_INVALID_ARG;
  muon_ctx* ctx = plan->ctx;
  if (plan->kind == PLAN_STATE8) return fail(ctx, MUON_ERR_INVALID_ARG, "the plan has no gradients");
  if (n != int32_t(plan->grads.size()) || (n > 0 && !grads))
    return fail(ctx, MUON_ERR_INVALID_ARG, "%d gradients for a plan of %zu tensors", n, plan->grads.size());
  for (const PlanBucket& b : plan->buckets)
    for (int i : b.tensors) {
      const uintptr_t lo = reinterpret_cast<uintptr_t>(grads[i]), hi = lo + uintptr_t(plan->grad_numel[i] * plan->grad_size[i]);
      if (lo == 0) return fail(ctx, MUON_ERR_INVALID_ARG, "tensor %d: NULL pointer", i);
      if (lo & uintptr_t(plan->grad_size[i] - 1))
        return fail(ctx, MUON_ERR_INVALID_ARG, "tensor %d: a pointer is not aligned to its element", i);
      // the first written span that ends past lo
      auto it = std::upper_bound(plan->written.begin(), plan->written.end(), lo,
                                 [](uintptr_t a, const std::pair<uintptr_t, uintptr_t>& w) { return a < w.second; });
      if (it != plan->written.end() && it->first < hi)
        return fail(ctx, MUON_ERR_INVALID_ARG, "tensor %d: the gradient overlaps a tensor that the step writes", i);
    }
  for (int i = 0; i < n; ++i) plan->grads[i] = grads[i];
  return MUON_OK;
}

muon_status muon_state8_plan_create(muon_ctx* ctx, const muon_state8_tensor* tensors, int32_t n, muon_plan** out) {
  return make_plan(ctx, out, PLAN_STATE8, [&](muon_plan* plan) -> muon_status {
    if (n < 0 || (n > 0 && !tensors)) return fail(ctx, MUON_ERR_INVALID_ARG, "bad tensor list");
    std::vector<Span> spans;
    std::vector<Q8Chunk> table;
    constexpr int64_t chunk = int64_t(STATE8_BLOCKS) * ST_WARPS * Q_BLOCK;
    size_t all = 0;
    for (int i = 0; i < n; ++i)
      if (tensors[i].numel > 0 && tensors[i].numel <= kMaxNumel) all += size_t(cdiv(tensors[i].numel, chunk));
    table.reserve(all);
    for (int i = 0; i < n; ++i) {
      const muon_state8_tensor& t = tensors[i];
      if (t.numel < 0 || t.numel > kMaxNumel)
        return fail(ctx, MUON_ERR_INVALID_ARG, "tensor %d: numel %lld", i, (long long)t.numel);
      if (t.value_dtype != MUON_F32 && t.value_dtype != MUON_BF16)
        return fail(ctx, MUON_ERR_INVALID_ARG, "tensor %d: value_dtype %d", i, t.value_dtype);
      if (t.second_moment != 0 && t.second_moment != 1)
        return fail(ctx, MUON_ERR_INVALID_ARG, "tensor %d: second_moment %d", i, t.second_moment);
      if (t.numel == 0) continue;
      if (!t.values || !t.codes || !t.scales) return fail(ctx, MUON_ERR_INVALID_ARG, "tensor %d: NULL pointer", i);
      if (!aligned_to(t.values, dtype_size(t.value_dtype)) || !aligned_to(t.scales, 4))
        return fail(ctx, MUON_ERR_INVALID_ARG, "tensor %d: a pointer is not aligned to its element", i);
      add_span(spans, t.values, t.numel * dtype_size(t.value_dtype), true);
      add_span(spans, t.codes, t.numel, true);
      add_span(spans, t.scales, cdiv(t.numel, Q_BLOCK) * 4, true);
      for (int64_t at = 0; at < t.numel; at += chunk) {
        Q8Chunk c{};
        c.values = static_cast<char*>(t.values) + at * dtype_size(t.value_dtype);
        c.codes = static_cast<char*>(t.codes) + at;
        c.scales = t.scales + at / Q_BLOCK;
        c.count = uint16_t(std::min<int64_t>(chunk, t.numel - at));
        c.second = uint8_t(t.second_moment);
        c.bf16 = t.value_dtype == MUON_BF16;
        table.push_back(c);
      }
    }
    if (overlapping(spans))
      return fail(ctx, MUON_ERR_INVALID_ARG, "two tensors of the plan overlap");
    plan->buckets.emplace_back();
    plan->buckets[0].chunks = table.size();
    CUDA_TRY(ctx, load_kernel(state8_kernel<true>));
    CUDA_TRY(ctx, load_kernel(state8_kernel<false>));
    return finish_plan(ctx, plan, table, out);
  });
}

static muon_status state8_run(muon_plan* plan, bool pack, void* stream) {
  muon_status s = check_plan(plan, PLAN_STATE8);
  if (s != MUON_OK) return s;
  muon_ctx* ctx = plan->ctx;
  const PlanBucket& b = plan->buckets[0];
  if (b.chunks == 0) return MUON_OK;
  DeviceGuard guard(plan->device);
  CUDA_TRY(ctx, guard.err);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  ctx->last_stream = st;
  CUDA_TRY(ctx, cudaGetLastError());
  ProfScope ps(ctx, MUON_K_OTHER, st);
  const Q8Chunk* t = static_cast<const Q8Chunk*>(plan->table);
  const dim3 grid{unsigned(b.chunks)};
  const int* flags = ctx->dflags;
  CUDA_TRY(ctx, pack ? launch_pdl(state8_kernel<true>, grid, dim3(ST_THREADS), size_t(0), st, t, flags)
                     : launch_pdl(state8_kernel<false>, grid, dim3(ST_THREADS), size_t(0), st, t, flags));
  ctx->launches++;
  return MUON_OK;
}

muon_status muon_state8_pack(muon_plan* plan, void* stream) { return state8_run(plan, true, stream); }

muon_status muon_state8_unpack(muon_plan* plan, void* stream) { return state8_run(plan, false, stream); }

void muon_plan_destroy(muon_plan* plan) {
  if (!plan) return;
  {
    std::lock_guard<std::mutex> lock(g_plans_mutex);
    if (plan->ctx) {
      auto& v = plan->ctx->plans;
      v.erase(std::remove(v.begin(), v.end(), plan), v.end());
    }
  }
  if (plan->table) {
    // cudaFree waits for work that may read the table.  Another stream may be
    // capturing just now: freeing must not end its capture.
    DeviceGuard guard(plan->device);
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    const bool relaxed = cudaThreadExchangeStreamCaptureMode(&mode) == cudaSuccess;
    cudaFree(plan->table);
    if (relaxed) cudaThreadExchangeStreamCaptureMode(&mode);
  }
  delete plan;
}

}  // extern "C"
