// What the stand-in launchers of the linear layer, the gated block and gradient
// clipping saw, and the fake device allocations they check against.
#pragma once
#include <cstdint>
#include <string>
#include <vector>

// Kernel instances launched since the last call, e.g. "tile256 cat a w^T".
std::vector<std::string> lin_stub_take();
void lin_stub_register(const void *p, int64_t bytes);
void lin_stub_reset();
// No names are kept (and nothing allocated) while quiet.
void lin_stub_quiet(bool on);
