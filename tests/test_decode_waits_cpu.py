"""Host check of the decode kernel's softmax role when a bounded wait gives up.  The eight softmax warps
meet at a named barrier in every tile, so a warp whose wait ran out must keep passing the barriers of the
others: a warp that left alone would strand them there for good.

`tc_softmax` and `tc_softmax_leave` are taken from the kernel's source as they stand and compiled for the host, a thread per warp
(its lane 0), with the PTX wrappers replaced by stand-ins: a wait gives up where the scenario says so (on
all warps, or on one, whose clock ran out first), and the named barrier reports a warp that is never joined.
"""
import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_latent_kv_20_b200", "csrc")

HOST = r"""
#include <algorithm>
#include <atomic>
#include <chrono>
#include <climits>
#include <cmath>
#include <condition_variable>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <mutex>
#include <set>
#include <string>
#include <thread>
#include <vector>
#define __device__
#define __forceinline__ inline
#define __noinline__
using std::max;
using std::min;
struct Dim { unsigned x; };
static thread_local Dim threadIdx;
static int warp_id() { return threadIdx.x >> 5; }
struct uint4 { uint32_t x, y, z, w; };
static uint4 make_uint4(uint32_t x, uint32_t y, uint32_t z, uint32_t w) { return {x, y, z, w}; }
struct __nv_bfloat16 { uint16_t v; };
struct __nv_bfloat162 { uint32_t v; };
static __nv_bfloat162 __floats2bfloat162_rn(float, float) { return {0}; }
static float __uint_as_float(uint32_t u) {
  float f;
  std::memcpy(&f, &u, 4);
  return f;
}
static bool __all_sync(unsigned, bool x) { return x; }   // one lane stands for its warp
static bool __any_sync(unsigned, bool x) { return x; }
static void __syncwarp() {}
constexpr int kHeads = 128, kDLat = 512;
constexpr float kLn2 = 0.6931471805599453f;
@CONSTANTS@
struct FullRows {
  static constexpr bool kHoles = false;
  struct Map {
    int real(int v) const { return v; }
    int hole0() const { return 0; }
    int hole1() const { return 0; }
  };
  Map map(int) const { return {}; }
};
struct Workspace { float *o, *m, *l; };
struct DecodeTcArgs {
  const int32_t* seq_lens;
  int capacity;
  float scale_log2;
  Workspace ws;
  __nv_bfloat16* out_lat;
  float* lse;
};
template <class Rows> static Rows tc_rows(const DecodeTcArgs&) { return {}; }
struct TcPlan { int start, end, b0, off0, b_end, len0; };
struct TcBars {
  uint64_t s_full[2], s_empty[2], p_full[2], p_empty[2], o_ready, o_final, o_free;
};
struct Segment { int b, tok_begin, tok_end, n_tiles; bool direct; int slot, len; };
static std::vector<int> segments;   // tiles of each
struct SegmentCursor {
  int b, off, start, end, b_end, pair;
  bool first;
  int len0;
  template <class Rows> bool next(const int32_t*, int, const Rows&, Segment& s) {
    if (b >= static_cast<int>(segments.size())) return false;
    s = {b, 0, segments[b] * kTcTile - 5, segments[b], true, 0, 0};
    ++b;
    return true;
  }
};

// --- the scenario: waits on the barriers `fail_bars` give up from their fail_from-th phase on, on warp
// fail_warp alone (or on all: -1)
static std::set<const void*> fail_bars;
static int fail_from, fail_warp;
static std::atomic<int> gave_up[8], late_arrivals, written;
static std::map<const void*, int> waited[8];
static bool mbar_wait(uint64_t* bar, uint32_t, uint32_t) {
  const int w = warp_id();
  if (gave_up[w] > 0) ++late_arrivals;   // a warp whose wait ran out waits for nothing more
  const int n = waited[w][bar]++;
  if (fail_bars.count(bar) == 0 || n < fail_from || (fail_warp >= 0 && w != fail_warp)) return true;
  ++gave_up[w];
  return false;
}
static TcBars bars;
static uint32_t smem_u32(const void* p) { return static_cast<uint32_t>(static_cast<const uint8_t*>(p) - reinterpret_cast<uint8_t*>(&bars)); }
static uint32_t mapa_shared(uint32_t a, uint32_t) { return a; }
static uint32_t lbar(const void* p) { return smem_u32(p); }
static std::mutex lock;
static std::map<uint32_t, int> arrivals;
static void mbar_arrive_relaxed(uint32_t a) {
  if (gave_up[warp_id()] > 0) ++late_arrivals;
  std::lock_guard<std::mutex> g(lock);
  ++arrivals[a];
}
static std::condition_variable cv;
static int inside = 0, phase = 0;
static void named_bar_sync(int, int) {
  std::unique_lock<std::mutex> g(lock);
  const int mine = phase;
  if (++inside == 8) {
    inside = 0;
    ++phase;
    cv.notify_all();
    return;
  }
  if (!cv.wait_for(g, std::chrono::seconds(3), [&] { return phase != mine; })) {
    std::printf("warp %d is stranded at the named barrier\n", warp_id());
    std::fflush(stdout);
    std::_Exit(3);
  }
}
static void tc_fence_before() {}
static void tc_fence_after() {}
static void fence_proxy_async_smem() {}
static void fence_release_smem_to_cluster() {}
static void tmem_ld_wait() {}
// Scores: the even warps' heads grow from tile to tile (they rescale O), the others' do not.
static thread_local int loads;
static void tmem_ld16(uint32_t, uint32_t (&r)[16]) {
  const float s = warp_id() % 2 == 0 ? 20.f * (loads / 2) : 1.f;
  ++loads;
  for (uint32_t& x : r) std::memcpy(&x, &s, 4);
}
static float ex2_approx(float x) { return std::exp2(x); }
static void tc_rescale_o(uint32_t, float) {}
static void tc_write_segment(bool, void*, float*, float*, uint8_t*, uint32_t, float, float) { ++written; }
template <bool kMapped, class Map>
static void tc_prefetch_tile(const DecodeTcArgs&, const Map&, int, int, int) {}

@SOFTMAX@

int main(int argc, char** argv) {
  const std::map<std::string, uint64_t*> names = {
      {"s_full0", &bars.s_full[0]}, {"s_full1", &bars.s_full[1]}, {"p_empty0", &bars.p_empty[0]},
      {"p_empty1", &bars.p_empty[1]}, {"o_ready", &bars.o_ready}, {"o_final", &bars.o_final}};
  for (const auto& n : names)
    if (std::string(argv[1]).find(n.first) != std::string::npos) fail_bars.insert(n.second);
  fail_from = std::atoi(argv[2]);
  fail_warp = std::atoi(argv[3]);
  for (int i = 4; i < argc; ++i) segments.push_back(std::atoi(argv[i]));
  static uint8_t smem[kTcSmemBytes];
  static float red[512], lse[64 * kHeads];
  static __nv_bfloat16 out[1];
  volatile int abort_flag = 0;
  const DecodeTcArgs a{nullptr, 0, 1.f, {nullptr, nullptr, nullptr}, out, lse};
  const TcPlan plan{0, 1, 0, 0, 1, 0};
  std::vector<std::thread> all;
  for (int w = 0; w < 8; ++w)
    all.emplace_back([&, w] {
      threadIdx.x = 32 * w;
      loads = 0;
      tc_softmax<false, FullRows>(a, plan, 0, smem, &bars, red, 0, 0, &abort_flag);
    });
  for (auto& t : all) t.join();
  int failed = 0, tiles = 0;
  for (int w = 0; w < 8; ++w) failed += gave_up[w] > 0;
  for (int n : segments) tiles += n;
  std::printf("failed %d abort %d late %d written %d s_empty %d p_full0 %d p_full1 %d tiles %d\n", failed, abort_flag != 0,
              late_arrivals.load(), written.load(), arrivals[smem_u32(&bars.s_empty[0])] + arrivals[smem_u32(&bars.s_empty[1])],
              arrivals[smem_u32(&bars.p_full[0])], arrivals[smem_u32(&bars.p_full[1])], tiles);
  return 0;
}
"""


def block(text, start):
    """The text from `start` to the end of the braces that follow it."""
    i = text.index(start)
    depth, j = 0, text.index("{", i)
    while True:
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        j += 1
        if depth == 0:
            return text[i:j]


@pytest.fixture(scope="module")
def softmax(tmp_path_factory):
    with open(os.path.join(CSRC, "decode_tc.cuh")) as f:
        src = f.read()
    constants = "\n".join(re.findall(r"^constexpr (?:int|uint32_t|float) kTc\w+ = [^;]*;", src, re.M))
    code = block(src, "template <class Rows>\n__device__ __noinline__ void tc_softmax_leave") + "\n" + block(
        src, "template <bool kMapped, class Rows>\n__device__ void tc_softmax(")
    where = tmp_path_factory.mktemp("softmax")
    cpp, exe = str(where / "softmax.cpp"), str(where / "softmax")
    with open(cpp, "w") as f:
        f.write(HOST.replace("@CONSTANTS@", constants).replace("@SOFTMAX@", code))
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-w", "-o", exe, cpp], check=True)

    def run(bar, first, warp, segments):
        p = subprocess.run([exe, bar, str(first), str(warp), *map(str, segments)], capture_output=True, text=True,
                           timeout=60)
        assert p.returncode == 0, p.stdout + p.stderr
        words = p.stdout.split()
        return dict(zip(words[::2], map(int, words[1::2])))

    return run


SEGMENTS = [5, 1, 3, 4]   # tiles of each


def test_without_a_timeout_every_tile_and_segment_is_done(softmax):
    r = softmax("none", 0, -1, SEGMENTS)
    assert r["failed"] == r["abort"] == r["late"] == 0
    assert r["written"] == 8 * len(SEGMENTS)
    assert r["s_empty"] == 8 * r["tiles"]
    assert r["p_full0"] == 8 * r["tiles"] and r["p_full1"] == 4 * r["tiles"]   # the second half's warps arrive twice


@pytest.mark.parametrize("warp", [-1, 0, 1, 5, 6])   # all, or the one whose limit ran out before the barrier completed
@pytest.mark.parametrize("first", [0, 1, 2])
# (a V copy that never lands leaves the second half of P taken and O unfinished)
@pytest.mark.parametrize("bar", ["s_full0", "s_full1", "p_empty0", "p_empty1", "o_ready", "o_final", "p_empty1+o_ready"])
def test_a_wait_that_gives_up_strands_no_warp(softmax, bar, first, warp):
    r = softmax(bar, first, warp, SEGMENTS)
    assert r["late"] == 0    # a warp that gave up neither waits nor arrives any more
    assert r["abort"] == (r["failed"] > 0)
    assert r["written"] < 8 * len(SEGMENTS) or r["failed"] == 0
