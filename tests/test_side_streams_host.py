"""The backwards' side streams (csrc/gla_side.cuh) against a fake of the runtime's calls, on the CPU: whichever
call fails, what was forked is joined; each device has a lock of its own; a pair inside another capture is
left alone."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "linear_attention_recurrence_simple_gb300", "csrc")

SOURCE = r"""
#include <cstdio>
#include <cstdlib>
#include <chrono>
#include <future>
#include <map>
#include <string>
#include <vector>
#include "gla_side.cuh"

struct Op { std::string what; long stream, event; };
static std::vector<Op> ops;
static long calls, fail_at, next_stream = 100, next_event = 1000, live_events;
static std::map<long, unsigned long long> capture;
static thread_local int current;

struct Fake {
  using Error = int;
  using Stream = long;
  using Event = long;
  static constexpr int kSuccess = 0, kInvalidDevice = 101;
  static int step(const char* what, long s, long ev) {
    if (calls++ == fail_at) return 7;
    ops.push_back({what, s, ev});
    return 0;
  }
  static int device(int& d) { d = current; return step("device", 0, 0); }
  static int capture_of(long s, unsigned long long& id) {
    id = capture.count(s) ? capture[s] : 0;
    return step("capture_of", s, 0);
  }
  static int create_pair(long (&s)[2]) {
    if (int e = step("create_pair", 0, 0)) return e;
    s[0] = next_stream++;
    s[1] = next_stream++;
    return 0;
  }
  static int create_event(long& ev) {
    if (int e = step("create_event", 0, 0)) return e;
    ev = next_event++;
    ++live_events;
    return 0;
  }
  static void destroy_event(long) { --live_events; }
  static int record(long ev, long s) { return step("record", s, ev); }
  static int wait(long s, long ev) { return step("wait", s, ev); }
  static void synchronize(long s) { ops.push_back({"synchronize", s, 0}); }
  static int launch(long s) { return step("launch", s, 0); }
};

#define CHECK(x) do { if (!(x)) { std::printf("line %d, call %ld fails: %s\n", __LINE__, fail_at, #x); std::exit(1); } } while (0)

static int backward(gla::SidePool<Fake>& pool, long stream) {
  gla::SideFork<Fake> f;
  int e = f.fork(pool, stream);
  if (!e) e = Fake::launch(f.side(0));
  if (!e) e = Fake::launch(f.side(1));
  if (!e) e = Fake::launch(stream);
  return f.join(e);
}

static void joined_whatever_fails() {
  fail_at = -1;
  calls = 0;
  {
    gla::SidePool<Fake> pool;
    CHECK(backward(pool, 5) == 0);
  }
  const long n = calls;
  for (fail_at = 0; fail_at < n; ++fail_at) {
    gla::SidePool<Fake> pool;
    calls = 0;
    ops.clear();
    CHECK(backward(pool, 5) == 7);
    CHECK(live_events == 0);
    // every side stream that waited for the call's stream is behind it again, after all that it was given
    std::map<long, int> last, back;
    std::map<long, long> recorded;
    for (int i = 0; i < (int)ops.size(); ++i) {
      const Op& o = ops[i];
      if (o.stream >= 100 && (o.what == "wait" || o.what == "launch")) last[o.stream] = i;
      if (o.what == "record") recorded[o.event] = o.stream;
      if (o.what == "wait" && o.stream == 5) back[recorded[o.event]] = i;
      if (o.what == "synchronize") back[o.stream] = i;
    }
    for (auto& s : last) CHECK(back.count(s.first) && back[s.first] > s.second);
    // and the lock is free
    const long was = fail_at;
    fail_at = -1;
    CHECK(backward(pool, 5) == 0);
    fail_at = was;
  }
  fail_at = -1;
}

static void a_lock_for_each_device() {
  fail_at = -1;
  gla::SidePool<Fake> pool;
  long s[2];
  std::unique_lock<std::mutex> hold;
  current = 0;
  CHECK(pool.take(5, s, hold) == 0);
  auto other = [&](int dev) {
    return std::async(std::launch::async, [&pool, dev] {
      current = dev;
      long t[2];
      std::unique_lock<std::mutex> h;
      return pool.take(6, t, h);
    });
  };
  auto on1 = other(1);
  CHECK(on1.wait_for(std::chrono::seconds(20)) == std::future_status::ready);
  CHECK(on1.get() == 0);
  auto on0 = other(0);
  CHECK(on0.wait_for(std::chrono::milliseconds(200)) == std::future_status::timeout);
  hold.unlock();
  CHECK(on0.get() == 0);
  current = 64;
  CHECK(pool.take(5, s, hold) == Fake::kInvalidDevice);
  current = 0;
}

static void captures() {
  fail_at = -1;
  gla::SidePool<Fake> pool;
  auto take = [&](long stream) {
    long s[2];
    std::unique_lock<std::mutex> hold;
    CHECK(pool.take(stream, s, hold) == 0);
    CHECK(s[1] == s[0] + 1);
    return s[0];
  };
  const long first = take(5);
  CHECK(take(6) == first);
  capture[5] = capture[first] = capture[first + 1] = 1;  // a capture of stream 5 took the pair
  CHECK(take(5) == first);
  const long second = take(6);                           // eager
  CHECK(second != first);
  capture[7] = 2;
  CHECK(take(7) == second);
  capture[second] = ~0ull;                               // that capture failed
  CHECK(take(6) != first && take(6) != second);
  capture.clear();
  CHECK(take(6) == first);
}

int main(int, char** argv) {
  const std::string what = argv[1];
  if (what == "join") joined_whatever_fails();
  if (what == "locks") a_lock_for_each_device();
  if (what == "captures") captures();
  std::printf("ok\n");
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("side")
    (d / "side.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", CSRC, "-o", str(d / "side"), str(d / "side.cpp")],
                   check=True)
    return str(d / "side")


@pytest.mark.parametrize("what", ["join", "locks", "captures"])
def test_side_streams(program, what):
    r = subprocess.run([program, what], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr
