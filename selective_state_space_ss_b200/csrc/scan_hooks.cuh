// scan_hooks.cuh -- the scan's test-hook settings and the state sizes it supports
// (host code of libssscan.so's first translation unit, ss_scan.cu)
#pragma once

#include <atomic>

namespace ssscan {
namespace {

// Test hooks (ss_scan_debug.h): consumed by the next ss_scan_fwd call.
std::atomic<long long> g_dbg_workers{0};
std::atomic<long long> g_dbg_skip_publish{-1};
std::atomic<long long> g_dbg_spin_limit{0};
std::atomic<long long> g_dbg_step_simple{0};
std::atomic<long long> g_dbg_segments{0};

bool supported_dstate(int n) { return n == 16 || n == 32 || n == 64 || n == 128; }

}  // namespace
}  // namespace ssscan
