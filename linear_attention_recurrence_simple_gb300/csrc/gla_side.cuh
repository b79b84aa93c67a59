// Side streams on which a call runs independent kernels beside its own stream's: forked from it and joined
// back with events.  Written over a struct of the runtime's calls, so that the host logic compiles and runs
// without a GPU.
#pragma once

#include <mutex>
#include <vector>

namespace gla {

// Pairs of side streams per device.  Eager calls use the first; a stream that joined a capture stays in
// it until the capture ends, so a call that meets a pair inside another capture takes the next one
// (created when there is none).
template <class Api>
class SidePool {
 public:
  using Error = typename Api::Error;
  using Stream = typename Api::Stream;
  static constexpr int kMaxDevices = 64;

  // The current device's pair for a call on `stream`.  `hold` is held until the caller has forked, filled
  // and joined the streams: a capture that took them in between would swallow an eager call's launches.
  // One lock per device: calls on different devices do not wait for one another.
  Error take(Stream stream, Stream (&out)[2], std::unique_lock<std::mutex>& hold) {
    int dev = 0;
    Error e = Api::device(dev);
    if (e != Api::kSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return Api::kInvalidDevice;
    unsigned long long mine = 0;
    if ((e = Api::capture_of(stream, mine)) != Api::kSuccess) return e;
    Device& d = devices_[dev];
    hold = std::unique_lock<std::mutex>(d.mu);
    for (const Pair& p : d.pairs) {
      bool fits = true;
      for (Stream s : p.s) {
        unsigned long long id = 0;
        if ((e = Api::capture_of(s, id)) != Api::kSuccess) return e;
        fits = fits && (id == 0 || id == mine);
      }
      if (fits) {
        out[0] = p.s[0];
        out[1] = p.s[1];
        return Api::kSuccess;
      }
    }
    Pair p = {};
    if ((e = Api::create_pair(p.s)) != Api::kSuccess) return e;
    d.pairs.push_back(p);
    out[0] = p.s[0];
    out[1] = p.s[1];
    return Api::kSuccess;
  }

 private:
  struct Pair {
    Stream s[2];
  };
  struct Device {
    std::mutex mu;
    std::vector<Pair> pairs;
  };
  Device devices_[kMaxDevices];
};

// One call's use of a pair: fork() makes both wait for the call's stream, join() makes the stream wait for
// both.
template <class Api>
class SideFork {
 public:
  using Error = typename Api::Error;
  using Stream = typename Api::Stream;
  using Event = typename Api::Event;

  Error fork(SidePool<Api>& pool, Stream stream) {
    stream_ = stream;
    Error e = pool.take(stream, side_, hold_);
    for (int i = 0; i < 3 && e == Api::kSuccess; ++i) e = Api::create_event(ev_[i]);
    if (e == Api::kSuccess) e = Api::record(ev_[2], stream_);
    for (int i = 0; i < 2 && e == Api::kSuccess; ++i) {
      e = Api::wait(side_[i], ev_[2]);
      forked_[i] = e == Api::kSuccess;
    }
    return e;
  }
  Stream side(int i) const { return side_[i]; }

  // Returns `e`, or the join's own first error.  Whatever failed before, a side stream that was forked is
  // joined: what was queued on it must not outlast the call unordered (the caller may free its buffers), nor
  // stay unjoined in a capture.  Where the join itself fails, the host waits for the stream.
  Error join(Error e) {
    for (int i = 0; i < 2; ++i) {
      if (!forked_[i]) continue;
      forked_[i] = false;
      Error j = Api::record(ev_[i], side_[i]);
      if (j == Api::kSuccess) j = Api::wait(stream_, ev_[i]);
      if (j != Api::kSuccess) Api::synchronize(side_[i]);
      if (e == Api::kSuccess) e = j;
    }
    for (int i = 0; i < 3; ++i)
      if (ev_[i]) {
        Api::destroy_event(ev_[i]);
        ev_[i] = Event();
      }
    if (hold_.owns_lock()) hold_.unlock();
    return e;
  }
  SideFork() = default;
  SideFork(const SideFork&) = delete;
  SideFork& operator=(const SideFork&) = delete;
  ~SideFork() { join(Api::kSuccess); }

 private:
  Stream stream_ = Stream();
  Stream side_[2] = {Stream(), Stream()};
  Event ev_[3] = {Event(), Event(), Event()};
  bool forked_[2] = {false, false};
  std::unique_lock<std::mutex> hold_;
};

#ifdef __CUDACC__
struct CudaSideApi {
  using Error = cudaError_t;
  using Stream = cudaStream_t;
  using Event = cudaEvent_t;
  static constexpr Error kSuccess = cudaSuccess, kInvalidDevice = cudaErrorInvalidDevice;

  static Error device(int& dev) { return cudaGetDevice(&dev); }
  // The capture that a stream is in: 0 none, ~0 one that has failed.
  static Error capture_of(Stream s, unsigned long long& id) {
    cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
    id = 0;
    const Error e = cudaStreamGetCaptureInfo(s, &st, &id);
    if (st == cudaStreamCaptureStatusNone) id = 0;
    if (st == cudaStreamCaptureStatusInvalidated) id = ~0ull;
    return e;
  }
  static Error create_pair(Stream (&s)[2]) {
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;  // (the caller may be capturing)
    Error e = cudaThreadExchangeStreamCaptureMode(&mode);
    if (e != cudaSuccess) return e;
    e = cudaStreamCreateWithFlags(&s[0], cudaStreamNonBlocking);
    if (e == cudaSuccess && (e = cudaStreamCreateWithFlags(&s[1], cudaStreamNonBlocking)) != cudaSuccess)
      cudaStreamDestroy(s[0]);
    cudaThreadExchangeStreamCaptureMode(&mode);
    return e;
  }
  static Error create_event(Event& ev) { return cudaEventCreateWithFlags(&ev, cudaEventDisableTiming); }
  static void destroy_event(Event ev) { cudaEventDestroy(ev); }
  static Error record(Event ev, Stream s) { return cudaEventRecord(ev, s); }
  static Error wait(Stream s, Event ev) { return cudaStreamWaitEvent(s, ev, 0); }
  static void synchronize(Stream s) { cudaStreamSynchronize(s); }
};

// The backwards' side streams.
inline SidePool<CudaSideApi>& side_pool() {
  static SidePool<CudaSideApi> pool;
  return pool;
}
#endif

}  // namespace gla
