// What the stand-in launchers of the vocabulary cross entropy and the AdamW step saw,
// and the fake device allocations they check against.
#pragma once
#include <cstdint>
#include <string>
#include <vector>

// Kernel instances launched since the last call, e.g. "tile256 stats a w^T".
std::vector<std::string> loss_stub_take();
void loss_stub_register(const void *p, int64_t bytes);
void loss_stub_reset();
// No names are kept (and nothing allocated) while quiet.
void loss_stub_quiet(bool on);
