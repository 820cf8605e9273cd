// Host helpers of the C entry points, shared by abi.cpp (which defines them) and
// grads.cpp: error messages, overlap and workspace checks, debugging switches.
#pragma once

#include <cstddef>
#include <cstdint>
#include <string>
#include <vector>

namespace dmuon {

int fail(int code, const std::string& msg);
void clear_error();

struct Range {
  uintptr_t lo, hi;
  bool ro;
};
int check_alias(std::vector<Range>& rs);
int check_workspace(void* ws, size_t have, size_t need);

// Per-call debugging switches (see call_env in abi.cpp).
struct CallEnv {
  int where = -3;     // -3 none, -2 plan, -1 table, else a phase id
  bool sync = false;  // DMUON_DEBUG_SYNC
};
CallEnv call_env();
int forced(const CallEnv& f, int where);
int settle(const CallEnv& f, void* stream, const char* what);
const char* phase_name(int phase);

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace dmuon
