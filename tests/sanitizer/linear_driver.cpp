// Drives the host code of the linear layer, the gated block and gradient
// clipping (validation, workspace sizes and offsets, the choice of kernel, tiles
// and splits) over random calls, built with AddressSanitizer and
// UndefinedBehaviorSanitizer and linked against the stand-in launchers of
// linear_stub.cpp, which check every range that a kernel would touch.  Device
// buffers are fake addresses.
//
//   driver            random calls; prints one summary line
//   driver nomem      every call again with each of its host allocations failing
//                     in turn: a status comes back, no exception
//   driver choose     reads lines "op dtype layout M K N odd" (op: linear,
//                     linear_bwd, gated, gated_bwd, with a - behind it without a workspace; odd: 1 takes operands off
//                     every vector alignment) and prints the kernels each call
//                     launches, joined by "; "
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
#include "linear_stub.h"

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

// Fake allocations, `skew` bytes off a 4 KiB boundary.
uintptr_t g_next = uintptr_t{1} << 44;
char *dev(int64_t bytes, int64_t skew = 0) {
  char *p = reinterpret_cast<char *>(g_next + static_cast<uintptr_t>(skew));
  lin_stub_register(p, bytes);
  g_next += ((static_cast<uintptr_t>(bytes + skew) + 4095) & ~uintptr_t{4095}) + 4096;
  return p;
}
void fresh() {
  lin_stub_reset();
  g_next = uintptr_t{1} << 44;
}

struct Case {
  int32_t dtype = TP_BF16, act = TP_ACT_SILU, layout = TP_WEIGHTS_MATH;
  int64_t M = 1, K = 1, N = 1;
  int64_t pad = 0, skew = 0;   // of rows (elements) and of buffers (elements)
  bool a = true, b = true, c = true;   // options (bias, residual, kept values; dX, dW, dbias)
  bool f32_out = false;
  int ws = 2;                  // 0 none (or the least), 1 one byte short, 2 what is asked for, 3 more
  int64_t es() const { return dtype == TP_F32 ? 4 : 2; }
  int64_t wr() const { return layout == TP_WEIGHTS_LINEAR ? N : K; }
  int64_t wc() const { return layout == TP_WEIGHTS_LINEAR ? K : N; }
  // A matrix of this case: rows cols + pad apart.
  char *mat(int64_t rows, int64_t cols, int64_t size) const {
    return dev(rows > 0 ? ((rows - 1) * (cols + pad) + cols) * size : 0, skew * size);
  }
};

int64_t give(int mode, int64_t asked, int64_t least) {
  return mode == 0 ? least : mode == 1 ? std::max(least, asked - 1) : mode == 2 ? asked : asked + 4096;
}

int run_linear(const Case& k) {
  tp_linear_args q{};
  q.dtype = k.dtype;
  q.act = k.act;
  q.weight_layout = k.layout;
  q.out_dtype = k.f32_out ? TP_F32 : k.dtype;
  q.M = k.M;
  q.N = k.N;
  q.K = k.K;
  int64_t asked = -1;
  expect(tp_linear_ws(&q, &asked) == TP_OK && asked >= 0, "tp_linear_ws");
  q.X = k.mat(k.M, k.K, k.es());
  q.X_ld = k.K + k.pad;
  q.W = k.mat(k.wr(), k.wc(), k.es());
  q.W_ld = k.wc() + k.pad;
  if (k.a) q.bias = reinterpret_cast<float *>(dev(k.N * 4, k.skew * 4));
  if (k.b) q.residual = k.mat(k.M, k.N, k.es());
  q.residual_ld = q.out_ld = q.pre_ld = k.N + k.pad;
  q.out = k.mat(k.M, k.N, k.f32_out ? 4 : k.es());
  if (k.c) q.pre_out = k.mat(k.M, k.N, k.es());
  q.ws_bytes = give(k.ws, asked, 0);
  q.ws = q.ws_bytes ? dev(q.ws_bytes) : nullptr;
  return tp_linear(&q, nullptr);
}

int run_linear_bwd(const Case& k) {
  tp_linear_bwd_args q{};
  q.dtype = k.dtype;
  q.act = k.act;
  q.weight_layout = k.layout;
  q.dx_dtype = q.dw_dtype = k.f32_out ? TP_F32 : k.dtype;
  q.accumulate = k.f32_out;
  q.M = k.M;
  q.N = k.N;
  q.K = k.K;
  q.X = k.mat(k.M, k.K, k.es());
  q.X_ld = k.K + k.pad;
  q.W = k.mat(k.wr(), k.wc(), k.es());
  q.W_ld = q.dW_ld = k.wc() + k.pad;
  q.dOut = k.mat(k.M, k.N, k.es());
  q.pre = k.mat(k.M, k.N, k.es());
  q.dOut_ld = q.pre_ld = k.N + k.pad;
  const int64_t oes = k.f32_out ? 4 : k.es();
  if (k.a) q.dX = k.mat(k.M, k.K, oes);
  q.dX_ld = k.K + k.pad;
  if (k.b) q.dW = k.mat(k.wr(), k.wc(), oes);
  if (k.c) q.dbias = reinterpret_cast<float *>(dev(k.N * 4, k.skew * 4));
  int64_t asked = -1;
  expect(tp_linear_backward_ws(&q, &asked) == TP_OK && asked >= 0, "tp_linear_backward_ws");
  // What it cannot do without: found by its refusals.
  int64_t least = 0;
  const bool keeps = k.act != TP_ACT_NONE && (k.a || k.b) && k.M > 0;
  if (keeps) least += (k.M * k.N * k.es() + 255) / 256 * 256;
  if (k.c) {
    tp_linear_bwd_args only = q;
    only.dX = only.dW = nullptr;
    int64_t n = 0;
    expect(tp_linear_backward_ws(&only, &n) == TP_OK, "tp_linear_backward_ws, dbias");
    least += n;
  }
  expect(least <= asked, "no more needed than asked for");
  if (least > 0) {
    q.ws_bytes = least - 1;
    q.ws = dev(least - 1);
    expect(tp_linear_backward(&q, nullptr) == TP_ERR_ARG, "a workspace too small");
  }
  q.ws_bytes = give(k.ws, asked, least);
  q.ws = q.ws_bytes ? dev(q.ws_bytes) : nullptr;
  lin_stub_take();
  return tp_linear_backward(&q, nullptr);
}

int run_gated(const Case& k) {
  tp_gated_args q{};
  q.dtype = k.dtype;
  q.act = k.act;
  q.weight_layout = k.layout;
  q.M = k.M;
  q.F = k.N;
  q.K = k.K;
  int64_t asked = -1;
  expect(tp_gated_linear_ws(&q, &asked) == TP_OK && asked >= 0, "tp_gated_linear_ws");
  q.X = k.mat(k.M, k.K, k.es());
  q.X_ld = k.K + k.pad;
  q.W_gate = k.mat(k.wr(), k.wc(), k.es());
  q.W_up = k.mat(k.wr(), k.wc(), k.es());
  q.W_ld = k.wc() + k.pad;
  q.out = k.mat(k.M, k.N, k.es());
  if (k.c) {
    q.gate_out = k.mat(k.M, k.N, k.es());
    q.up_out = k.mat(k.M, k.N, k.es());
  }
  q.out_ld = q.keep_ld = k.N + k.pad;
  q.ws_bytes = give(k.ws, asked, 0);
  q.ws = q.ws_bytes ? dev(q.ws_bytes) : nullptr;
  return tp_gated_linear(&q, nullptr);
}

int run_gated_bwd(const Case& k) {
  tp_gated_bwd_args q{};
  q.dtype = k.dtype;
  q.act = k.act;
  q.weight_layout = k.layout;
  q.dx_dtype = q.dw_dtype = k.f32_out ? TP_F32 : k.dtype;
  q.accumulate = k.f32_out;
  q.M = k.M;
  q.F = k.N;
  q.K = k.K;
  int64_t asked = -1;
  expect(tp_gated_linear_backward_ws(&q, &asked) == TP_OK && asked >= 0, "tp_gated_linear_backward_ws");
  q.X = k.mat(k.M, k.K, k.es());
  q.X_ld = k.K + k.pad;
  q.W_gate = k.mat(k.wr(), k.wc(), k.es());
  q.W_up = k.mat(k.wr(), k.wc(), k.es());
  q.W_ld = q.dW_ld = k.wc() + k.pad;
  q.gate = k.mat(k.M, k.N, k.es());
  q.up = k.mat(k.M, k.N, k.es());
  q.dOut = k.mat(k.M, k.N, k.es());
  q.keep_ld = q.dOut_ld = k.N + k.pad;
  const int64_t oes = k.f32_out ? 4 : k.es();
  if (k.a) q.dX = k.mat(k.M, k.K, oes);
  q.dX_ld = k.K + k.pad;
  if (k.b) {
    q.dW_gate = k.mat(k.wr(), k.wc(), oes);
    q.dW_up = k.mat(k.wr(), k.wc(), oes);
  }
  const int64_t least = 2 * ((k.M * k.N * k.es() + 255) / 256 * 256);
  expect(least <= asked, "no more needed than asked for");
  if (least > 0) {
    q.ws_bytes = least - 1;
    q.ws = dev(least - 1);
    expect(tp_gated_linear_backward(&q, nullptr) == TP_ERR_ARG, "a workspace too small");
  }
  q.ws_bytes = give(k.ws, asked, least);
  q.ws = q.ws_bytes ? dev(q.ws_bytes) : nullptr;
  lin_stub_take();
  return tp_gated_linear_backward(&q, nullptr);
}

int run(const std::string& op, const Case& k) {
  fresh();
  lin_stub_take();
  if (op == "linear") return run_linear(k);
  if (op == "linear_bwd") return run_linear_bwd(k);
  if (op == "gated") return run_gated(k);
  if (op == "gated_bwd") return run_gated_bwd(k);
  expect(false, "unknown op");
  return 0;
}

int choose() {
  std::string op, dtype, layout;
  Case k;
  int odd;
  while (std::cin >> op >> dtype >> layout >> k.M >> k.K >> k.N >> odd) {
    k.dtype = dtype == "f32" ? TP_F32 : TP_BF16;
    k.layout = layout == "linear" ? TP_WEIGHTS_LINEAR : TP_WEIGHTS_MATH;
    k.pad = k.skew = odd;
    k.ws = op.back() == '-' ? 0 : 2;
    if (!k.ws) op.pop_back();
    expect(run(op, k) == TP_OK, "a call to choose for");
    const auto names = lin_stub_take();
    for (size_t i = 0; i < names.size(); ++i) std::printf("%s%s", i ? "; " : "", names[i].c_str());
    std::printf("\n");
  }
  return 0;
}

// A far call: sizes at the edge of what is taken, or past it.
void limits() {
  const int64_t big[] = {int64_t{1} << 20, (int64_t{1} << 26) - 1, int64_t{1} << 26, (int64_t{1} << 31) - 1, int64_t{1} << 31, int64_t{1} << 40};
  long taken = 0, refused = 0;
  for (const char *op : {"linear", "linear_bwd", "gated", "gated_bwd"})
    for (int64_t v : big)
      for (int which = 0; which < 3; ++which) {
        Case k;
        (which == 0 ? k.M : which == 1 ? k.K : k.N) = v;
        tp_linear_args q{};
        q.dtype = k.dtype;
        q.M = k.M;
        q.N = k.N;
        q.K = k.K;
        int64_t n = 0;
        if (tp_linear_ws(&q, &n) != TP_OK) {
          ++refused;
          continue;
        }
        expect(run(op, k) == TP_OK, "a far call");
        ++taken;
      }
  expect(taken > 20 && refused > 20, "calls on both sides of the limits");
}

void grads(std::mt19937& rng) {
  for (int i = 0; i < 300; ++i) {
    fresh();
    const int num = static_cast<int>(rng() % 200);
    std::vector<tp_grad_tensor> ts;
    for (int j = 0; j < num; ++j) {
      tp_grad_tensor t{};
      t.dtype = rng() % 2 ? TP_F32 : TP_BF16;
      t.n = rng() % 4 ? static_cast<int64_t>(rng() % 20000) : 0;
      const int64_t es = t.dtype == TP_F32 ? 4 : 2;
      t.grad = t.n ? dev(t.n * es, es) : nullptr;
      t.out = rng() % 2 ? const_cast<void *>(t.grad) : t.n ? dev(t.n * es) : nullptr;
      ts.push_back(t);
    }
    const int64_t ranks = 1 + rng() % 64;
    auto *parts = reinterpret_cast<double *>(dev(ranks * TP_GRAD_PARTS * 8));
    auto *norm = rng() % 2 ? reinterpret_cast<float *>(dev(4)) : nullptr;
    expect(tp_grad_sumsq(ts.data(), num, parts, nullptr) == TP_OK, "sum of squares");
    expect(tp_grad_clip(ts.data(), num, parts, ranks, 1.0, 1e-6, norm, nullptr) == TP_OK, "clipping");
    expect(tp_grad_clip(ts.data(), num, parts, 65, 1.0, 1e-6, norm, nullptr) == TP_ERR_ARG, "ranks");
    for (size_t a = 0; a < ts.size(); ++a)      // an output over another gradient
      if (ts[a].n && a + 1 < ts.size() && ts[a + 1].n) {
        auto bad = ts;
        bad[a].dtype = bad[a + 1].dtype;
        bad[a].n = std::min(bad[a].n, bad[a + 1].n);
        bad[a].grad = bad[a + 1].out;
        bad[a].out = bad[a + 1].out;
        expect(tp_grad_clip(bad.data(), num, parts, ranks, 1.0, 1e-6, norm, nullptr) == TP_ERR_ARG, "outputs overlap");
        break;
      }
  }
}

// f() with its n-th allocation failing, for every n.
template <typename F>
long starve(F&& f) {
  long failed = 0;
  for (long n = 0; n < 1000; ++n) {
    int rc;
    lin_stub_quiet(true);
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
    lin_stub_quiet(false);
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
  char *p = dev(1 << 22), *o = dev(1 << 22);
  auto at = [&](int i) { return p + i * (1 << 16); };
  long failed = 0;
  for (bool good : {true, false}) {      // a valid call, and one refused with a long message
    tp_linear_args l{};
    l.dtype = l.out_dtype = TP_BF16;
    l.M = 32;
    l.N = l.K = 64;
    l.X = at(0);
    l.W = at(1);
    l.bias = reinterpret_cast<float *>(at(2));
    l.residual = at(3);
    l.out = good ? at(4) : at(0);
    failed += starve([&] { return tp_linear(&l, nullptr); });
    tp_linear_bwd_args b{};
    b.dtype = b.dx_dtype = b.dw_dtype = TP_BF16;
    b.act = TP_ACT_SILU;
    b.M = 32;
    b.N = b.K = 64;
    b.X = at(0);
    b.W = at(1);
    b.dOut = at(2);
    b.pre = at(3);
    b.dX = good ? at(4) : at(0);
    b.dW = at(5);
    b.dbias = reinterpret_cast<float *>(at(6));
    b.ws = o;
    b.ws_bytes = 1 << 22;
    failed += starve([&] { return tp_linear_backward(&b, nullptr); });
    tp_gated_args g{};
    g.dtype = TP_BF16;
    g.M = 32;
    g.F = g.K = 64;
    g.X = at(0);
    g.W_gate = at(1);
    g.W_up = at(2);
    g.out = good ? at(3) : at(0);
    failed += starve([&] { return tp_gated_linear(&g, nullptr); });
    tp_gated_bwd_args q{};
    q.dtype = q.dx_dtype = q.dw_dtype = TP_BF16;
    q.M = 32;
    q.F = q.K = 64;
    q.X = at(0);
    q.W_gate = at(1);
    q.W_up = at(2);
    q.gate = at(3);
    q.up = at(4);
    q.dOut = at(5);
    q.dX = good ? at(6) : at(0);
    q.dW_gate = at(7);
    q.dW_up = at(8);
    q.ws = o;
    q.ws_bytes = 1 << 22;
    failed += starve([&] { return tp_gated_linear_backward(&q, nullptr); });
    std::vector<tp_grad_tensor> ts;
    for (int i = 0; i < 40; ++i) ts.push_back({at(i), good ? at(i) : at(0), 100, TP_F32});
    auto *parts = reinterpret_cast<double *>(o);
    failed += starve([&] { return tp_grad_sumsq(ts.data(), 40, parts, nullptr); });
    failed += starve([&] { return tp_grad_clip(ts.data(), 40, parts, 2, 1.0, 1e-6, nullptr, nullptr); });
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
  long calls = 0, split = 0;
  auto size = [&](double lo, double hi) {
    const double u = std::uniform_real_distribution<double>(std::log(lo), std::log(hi))(rng);
    auto v = static_cast<int64_t>(std::exp(u) + 0.5);
    if (rng() % 2 && v >= 32) v = v / 32 * 32;
    if (rng() % 4 == 0 && v >= 64) v = v / 64 * 64;
    return std::max<int64_t>(1, v);
  };
  for (int i = 0; i < 40000; ++i) {
    Case k;
    k.dtype = rng() % 3 ? TP_BF16 : TP_F32;
    k.act = static_cast<int32_t>(rng() % 5);
    k.layout = rng() % 2 ? TP_WEIGHTS_MATH : TP_WEIGHTS_LINEAR;
    k.M = rng() % 3 ? size(1, 20000) : rng() % 8 == 0 ? 0 : size(1, 80);
    k.K = size(1, 30000);
    k.N = size(1, 30000);
    if (rng() % 3 == 0) k.pad = static_cast<int64_t>(rng() % 17);
    if (rng() % 4 == 0) k.pad = 8 * static_cast<int64_t>(rng() % 17);
    if (rng() % 4 == 0) k.skew = static_cast<int64_t>(rng() % 9);
    k.a = rng() % 2;
    k.b = rng() % 2;
    k.c = rng() % 2;
    k.f32_out = rng() % 3 == 0;
    k.ws = static_cast<int>(rng() % 4);
    for (const char *op : {"linear", "linear_bwd", "gated", "gated_bwd"}) {
      const int rc = run(op, k);
      expect(rc == TP_OK, "a valid call");
      ++calls;
      for (const std::string& s : lin_stub_take()) {
        kernels.insert(s);
        split += s.size() > 6 && s.substr(s.size() - 6) == " split";
      }
    }
  }
  limits();
  grads(rng);
  std::printf("calls %ld split %ld kernels %ld\n", calls, split, static_cast<long>(kernels.size()));
  for (const std::string& s : kernels) std::fprintf(stderr, "%s\n", s.c_str());
  return 0;
}
