// Drives the host code of the vocabulary cross entropy and the AdamW step (validation,
// workspace sizes and offsets, pieces, the choice of kernel, tiles and splits) over
// random calls, built with AddressSanitizer and UndefinedBehaviorSanitizer and linked
// against the stand-in launchers of loss_stub.cpp, which check every range that a
// kernel would touch.  Device buffers are fake addresses.
//
//   driver            random calls; prints a summary line, and the kernels on stderr
//   driver nomem      calls with each of their host allocations failing in turn
//   driver choose     reads lines "op dtype layout M K V odd piece" (op: ce, ce_bwd; odd: 1
//                     takes operands off every vector alignment) and prints the kernels
//                     each call launches, joined by "; "
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <iostream>
#include <new>
#include <random>
#include <set>
#include <string>
#include <vector>

#include "../../include/tpshard.h"
#include "loss_stub.h"

namespace {
long g_allocs_left = -1;   // allocations until one fails (-1: none does)
}

void *operator new(std::size_t n) {
  if (g_allocs_left >= 0 && g_allocs_left-- == 0) throw std::bad_alloc();
  if (void *p = std::malloc(n ? n : 1)) return p;
  throw std::bad_alloc();
}
void operator delete(void *p) noexcept { std::free(p); }
void operator delete(void *p, std::size_t) noexcept { std::free(p); }

namespace {

void expect(bool ok, const char *what) {
  if (ok) return;
  std::fprintf(stderr, "check failed: %s (last error: %s)\n", what, tp_last_error());
  std::abort();
}

uintptr_t g_next = uintptr_t{1} << 44;
char *dev(int64_t bytes, int64_t skew = 0) {
  char *p = reinterpret_cast<char *>(g_next + static_cast<uintptr_t>(skew));
  loss_stub_register(p, bytes);
  g_next += ((static_cast<uintptr_t>(bytes + skew) + 4095) & ~uintptr_t{4095}) + 4096;
  return p;
}
template <typename T>
T *dev_of(int64_t n, int64_t skew = 0) { return reinterpret_cast<T *>(dev(n * static_cast<int64_t>(sizeof(T)), skew * static_cast<int64_t>(sizeof(T)))); }
void fresh() {
  loss_stub_reset();
  g_next = uintptr_t{1} << 44;
}

struct Case {
  int32_t dtype = TP_BF16, layout = TP_WEIGHTS_MATH;
  int64_t M = 1, K = 1, V = 1, begin = 0, piece = 0;
  int64_t pad = 0, skew = 0;   // of rows and of buffers (elements)
  bool a = true, b = true, c = true;   // stats, loss, lse; dX, dW, dlse
  bool f32_out = false;
  int64_t es() const { return dtype == TP_F32 ? 4 : 2; }
  int64_t wr() const { return layout == TP_WEIGHTS_LINEAR ? V : K; }
  int64_t wc() const { return layout == TP_WEIGHTS_LINEAR ? K : V; }
  char *mat(int64_t rows, int64_t cols, int64_t size) const {
    return dev(rows > 0 ? ((rows - 1) * (cols + pad) + cols) * size : 0, skew * size);
  }
};

int run_ce(const Case& k) {
  tp_linear_ce_args q{};
  q.dtype = k.dtype;
  q.weight_layout = k.layout;
  q.M = k.M;
  q.V = k.V;
  q.K = k.K;
  int64_t asked = -1;
  expect(tp_linear_ce_ws(&q, &asked) == TP_OK && asked >= 0, "tp_linear_ce_ws");
  q.X = k.mat(k.M, k.K, k.es());
  q.X_ld = k.K + k.pad;
  q.W = k.mat(k.wr(), k.wc(), k.es());
  q.W_ld = k.wc() + k.pad;
  q.targets = dev_of<int64_t>(k.M, k.skew);
  q.vocab_begin = k.begin;
  q.ignore_index = -100;
  if (k.a) q.stats = dev_of<float>(3 * k.M, k.skew);
  if (k.b) q.loss = dev_of<float>(k.M, k.skew);
  if (k.c || !(k.a || k.b)) q.lse = dev_of<float>(k.M, k.skew);
  if (asked > 0) {
    q.ws_bytes = asked - 1;
    q.ws = dev(asked - 1);
    expect(tp_linear_ce(&q, nullptr) == TP_ERR_ARG, "a workspace too small");
  }
  q.ws_bytes = asked;
  q.ws = asked ? dev(asked) : nullptr;
  loss_stub_take();
  return tp_linear_ce(&q, nullptr);
}

int run_ce_bwd(const Case& k) {
  tp_linear_ce_bwd_args q{};
  q.dtype = k.dtype;
  q.weight_layout = k.layout;
  q.dx_dtype = q.dw_dtype = k.f32_out ? TP_F32 : k.dtype;
  q.accumulate = k.f32_out;
  q.M = k.M;
  q.V = k.V;
  q.K = k.K;
  q.piece = k.piece;
  q.X = k.mat(k.M, k.K, k.es());
  q.X_ld = q.dX_ld = k.K + k.pad;
  q.W = k.mat(k.wr(), k.wc(), k.es());
  q.W_ld = q.dW_ld = k.wc() + k.pad;
  q.targets = dev_of<int64_t>(k.M, k.skew);
  q.vocab_begin = k.begin;
  q.lse = dev_of<float>(k.M, k.skew);
  q.dloss_stride = k.c;
  q.dloss = dev_of<float>(k.c ? k.M : 1);
  q.dlse_stride = !k.c;
  if (k.b) q.dlse = dev_of<float>(k.c ? 1 : k.M);
  const int64_t oes = k.f32_out ? 4 : k.es();
  if (k.a) q.dX = k.mat(k.M, k.K, oes);
  if (k.b || !k.a) q.dW = k.mat(k.wr(), k.wc(), oes);
  int64_t asked = -1;
  expect(tp_linear_ce_backward_ws(&q, &asked) == TP_OK && asked > 0, "tp_linear_ce_backward_ws");
  q.ws_bytes = asked - 1;
  q.ws = dev(asked - 1);
  expect(tp_linear_ce_backward(&q, nullptr) == TP_ERR_ARG, "a workspace too small");
  q.ws_bytes = asked;
  q.ws = dev(asked);
  loss_stub_take();
  return tp_linear_ce_backward(&q, nullptr);
}

int run(const std::string& op, const Case& k) {
  fresh();
  loss_stub_take();
  if (op == "ce") return run_ce(k);
  expect(op == "ce_bwd", "unknown op");
  return run_ce_bwd(k);
}

int choose() {
  std::string op, dtype, layout;
  Case k;
  int odd;
  while (std::cin >> op >> dtype >> layout >> k.M >> k.K >> k.V >> odd >> k.piece) {
    k.dtype = dtype == "f32" ? TP_F32 : TP_BF16;
    k.layout = layout == "linear" ? TP_WEIGHTS_LINEAR : TP_WEIGHTS_MATH;
    k.pad = k.skew = odd;
    expect(run(op, k) == TP_OK, "a call to choose for");
    const auto names = loss_stub_take();
    for (size_t i = 0; i < names.size(); ++i) std::printf("%s%s", i ? "; " : "", names[i].c_str());
    std::printf("\n");
  }
  return 0;
}

// Sizes at the edge of what is taken, or past it.
void limits() {
  const int64_t big[] = {int64_t{1} << 18, int64_t{1} << 20, (int64_t{1} << 24) - 1, int64_t{1} << 24, int64_t{1} << 26, (int64_t{1} << 31) - 1, int64_t{1} << 31,
                         int64_t{1} << 40};
  long taken = 0, refused = 0;
  for (const char *op : {"ce", "ce_bwd"})
    for (int layout = 0; layout < 2; ++layout)
      for (int64_t v : big)
        for (int which = 0; which < 3; ++which) {
          Case k;
          k.layout = layout;
          k.M = k.K = k.V = 64;
          (which == 0 ? k.M : which == 1 ? k.K : k.V) = v;
          tp_linear_ce_args q{};
          q.dtype = k.dtype;
          q.M = k.M;
          q.V = k.V;
          q.K = k.K;
          int64_t n = 0;
          if (tp_linear_ce_ws(&q, &n) != TP_OK) {
            ++refused;
            continue;
          }
          expect(run(op, k) == TP_OK, "a far call");
          ++taken;
        }
  expect(taken > 20 && refused > 20, "calls on both sides of the limits");
}

struct Adam {
  std::vector<tp_adamw_tensor> ts;
  tp_adamw_args a{};
};
Adam adam(std::mt19937& rng, int num, bool codes) {
  Adam r;
  for (int j = 0; j < num; ++j) {
    tp_adamw_tensor t{};
    t.param_dtype = rng() % 2 ? TP_F32 : TP_BF16;
    t.grad_dtype = rng() % 2 ? TP_F32 : TP_BF16;
    t.n = rng() % 4 ? static_cast<int64_t>(rng() % (rng() % 16 ? 20000 : 10000000)) : 0;
    if (t.n) {
      const int64_t skew = static_cast<int64_t>(rng() % 3), scales = (t.n + TP_ADAMW_BLOCK - 1) / TP_ADAMW_BLOCK;
      t.param = dev(t.n * (t.param_dtype == TP_F32 ? 4 : 2), 4 * skew);
      t.grad = dev(t.n * (t.grad_dtype == TP_F32 ? 4 : 2), 4 * skew);
      t.m = dev(t.n * (codes ? 1 : 4), codes ? skew : 4 * skew);
      t.v = dev(t.n * (codes ? 1 : 4), codes ? skew : 4 * skew);
      if (codes) t.m_scale = dev_of<float>(scales, skew);
      if (codes) t.v_scale = dev_of<float>(scales, skew);
      if (rng() % 2) t.copy = dev(t.n * 2, 2 * skew);
    }
    r.ts.push_back(t);
  }
  r.a.states = codes ? TP_ADAMW_8BIT : TP_ADAMW_F32;
  r.a.lr = 1e-3;
  r.a.beta1 = 0.9;
  r.a.beta2 = 0.999;
  r.a.step = 1;
  if (rng() % 2) {
    r.a.ranks = 1 + rng() % 64;
    r.a.parts = dev_of<double>(r.a.ranks * TP_GRAD_PARTS);
    r.a.max_norm = 1.0;
    if (rng() % 2) r.a.norm_out = dev_of<float>(1);
  }
  if (rng() % 2) r.a.step_dev = dev_of<int64_t>(1);
  if (rng() % 2) r.a.lr_dev = dev_of<float>(1);
  return r;
}
void adams(std::mt19937& rng) {
  for (int i = 0; i < 400; ++i) {
    fresh();
    const bool codes = rng() % 2;
    Adam r = adam(rng, static_cast<int>(rng() % 120), codes);
    const int64_t num = static_cast<int64_t>(r.ts.size());
    expect(tp_adamw_step(r.ts.data(), num, &r.a, nullptr) == TP_OK, "a step");
    std::vector<tp_adamw_state> st;
    for (const auto& t : r.ts)
      if (codes) st.push_back({t.m, t.v, t.m_scale, t.v_scale, t.n ? dev(t.n * 2) : nullptr, t.n ? dev(t.n * 2) : nullptr, t.n, TP_BF16});
    expect(tp_adamw_unpack(st.data(), static_cast<int64_t>(st.size()), nullptr) == TP_OK, "states");
    for (int64_t j = 0; j + 1 < num; ++j)      // one tensor's weights over the next one's state
      if (r.ts[j].n && r.ts[j + 1].n) {
        Adam bad = r;
        bad.ts[j].param = bad.ts[j + 1].m;
        bad.ts[j].param_dtype = TP_BF16;
        if (reinterpret_cast<uintptr_t>(bad.ts[j].param) % 2 == 0)
          expect(tp_adamw_step(bad.ts.data(), num, &bad.a, nullptr) == TP_ERR_ARG, "buffers overlap");
        break;
      }
  }
}

template <typename F>
long starve(F&& f) {
  long failed = 0;
  for (long n = 0; n < 1000; ++n) {
    int rc;
    loss_stub_quiet(true);
    g_allocs_left = n;
    try {
      rc = f();
    } catch (...) {
      g_allocs_left = -1;
      std::fprintf(stderr, "an exception left a C entry (allocation %ld)\n", n);
      std::abort();
    }
    const bool hit = g_allocs_left < 0;
    g_allocs_left = -1;
    loss_stub_quiet(false);
    if (!hit) {
      expect(rc == TP_OK || rc == TP_ERR_ARG, "a call with memory");
      return failed;
    }
    ++failed;
    expect(rc == TP_ERR_HIP || rc == TP_ERR_ARG, "a call without memory");
    expect(std::strlen(tp_last_error()) > 0, "its message");
  }
  return failed;
}

int nomem() {
  fresh();
  std::mt19937 rng(7);
  long failed = 0;
  for (bool good : {true, false}) {
    tp_linear_ce_args q{};
    q.dtype = TP_BF16;
    q.M = q.V = q.K = 64;
    int64_t n = 0;
    expect(tp_linear_ce_ws(&q, &n) == TP_OK, "ws");
    q.X = dev(64 * 64 * 2);
    q.W = dev(64 * 64 * 2);
    q.targets = dev_of<int64_t>(64);
    q.loss = good ? dev_of<float>(64) : reinterpret_cast<float *>(const_cast<void *>(q.X));
    q.ws = dev(n);
    q.ws_bytes = n;
    failed += starve([&] { return tp_linear_ce(&q, nullptr); });
    failed += starve([&] { return tp_ce_join(reinterpret_cast<const float *>(q.X), 1, 64, q.targets, 0, q.loss, nullptr, nullptr); });
    tp_linear_ce_bwd_args b{};
    b.dtype = b.dx_dtype = b.dw_dtype = TP_BF16;
    b.M = b.V = b.K = 64;
    b.X = q.X;
    b.W = q.W;
    b.targets = q.targets;
    b.lse = dev_of<float>(64);
    b.dX = good ? dev(64 * 64 * 2) : const_cast<void *>(q.X);
    b.dW = dev(64 * 64 * 2);
    expect(tp_linear_ce_backward_ws(&b, &n) == TP_OK, "ws");
    b.ws = dev(n);
    b.ws_bytes = n;
    failed += starve([&] { return tp_linear_ce_backward(&b, nullptr); });
    Adam r = adam(rng, 60, true);
    if (!good) r.ts[3].n = -1;
    failed += starve([&] { return tp_adamw_step(r.ts.data(), 60, &r.a, nullptr); });
    std::vector<tp_adamw_state> st;
    for (int i = 0; i < 50; ++i) st.push_back({dev(100), dev(100), dev_of<float>(1), dev_of<float>(1), dev(400), dev(400), good ? 100 : -1, TP_F32});
    failed += starve([&] { return tp_adamw_unpack(st.data(), 50, nullptr); });
  }
  std::printf("failed %ld\n", failed);
  return 0;
}

}  // namespace

int main(int argc, char **argv) {
  if (argc > 1 && !std::strcmp(argv[1], "choose")) return choose();
  if (argc > 1 && !std::strcmp(argv[1], "nomem")) return nomem();
  std::mt19937 rng(1);
  std::set<std::string> kernels;
  long calls = 0;
  auto size = [&](double lo, double hi) {
    const double u = std::uniform_real_distribution<double>(std::log(lo), std::log(hi))(rng);
    auto v = static_cast<int64_t>(std::exp(u) + 0.5);
    if (rng() % 2 && v >= 32) v = v / 32 * 32;
    if (rng() % 4 == 0 && v >= 64) v = v / 64 * 64;
    return std::max<int64_t>(1, v);
  };
  for (int i = 0; i < 12000; ++i) {
    Case k;
    k.dtype = rng() % 3 ? TP_BF16 : TP_F32;
    k.layout = rng() % 2 ? TP_WEIGHTS_MATH : TP_WEIGHTS_LINEAR;
    k.M = rng() % 3 ? size(1, 40000) : rng() % 8 == 0 ? 0 : size(1, 80);
    k.K = size(1, 30000);
    k.V = size(1, 600000);
    k.begin = static_cast<int64_t>(rng());
    k.piece = rng() % 3 ? 0 : size(1, 100000);
    if (rng() % 3 == 0) k.pad = static_cast<int64_t>(rng() % 17);
    if (rng() % 4 == 0) k.pad = 8 * static_cast<int64_t>(rng() % 17);
    if (rng() % 4 == 0) k.skew = static_cast<int64_t>(rng() % 9);
    k.a = rng() % 2;
    k.b = rng() % 2;
    k.c = rng() % 2;
    k.f32_out = rng() % 3 == 0;
    for (const char *op : {"ce", "ce_bwd"}) {
      expect(run(op, k) == TP_OK, "a valid call");
      ++calls;
      for (const std::string& s : loss_stub_take()) kernels.insert(s);
    }
  }
  limits();
  adams(rng);
  for (const std::string& s : loss_stub_take()) kernels.insert(s);
  std::printf("calls %ld kernels %ld\n", calls, static_cast<long>(kernels.size()));
  for (const std::string& s : kernels) std::fprintf(stderr, "%s\n", s.c_str());
  return 0;
}
