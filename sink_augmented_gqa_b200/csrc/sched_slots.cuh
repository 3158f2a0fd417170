// Counter slots of the prefill kernel's dynamic schedule (g_prefill_sched:
// one counter pair per slot, reset by the last CTA of the launch that used
// it). Two launches in flight at once must never share a slot.
//  * Launches made outside stream capture take slots [0, kEagerSchedSlots)
//    round robin. Before one reuses a slot its stream waits for the event
//    recorded after the slot's previous launch, so the two are ordered
//    whatever streams they run on (normally that launch finished long ago
//    and the wait costs nothing).
//  * Launches captured into a CUDA graph cannot wait on work outside the
//    capture; they take slots [kEagerSchedSlots, kEagerSchedSlots +
//    kGraphSchedSlots) round robin, so a graph never shares a slot with an
//    eager launch. Graph replays that overlap one another must not hold more
//    than kGraphSchedSlots prefill launches between them.
// Host code only; Api stands for the CUDA runtime (sinkattn.cu), or for a fake
// of it whose calls fail.
#pragma once

#include <mutex>
#include <stdint.h>

namespace sa {

constexpr int kEagerSchedSlots = 64;
constexpr int kGraphSchedSlots = 64;

inline int sched_slot_of(uint64_t index, bool captured) {
  return captured ? kEagerSchedSlots + (int)(index % kGraphSchedSlots) : (int)(index % kEagerSchedSlots);
}

// One device's slots. Api: types Status, Stream, Event (null when {}); kOk;
// create(Event*), wait(Stream, Event), record(Event, Stream) return a Status.
template <typename Api>
struct SchedSlots {
  std::mutex mu;
  uint64_t eager_next = 0, graph_next = 0;
  typename Api::Event done[kEagerSchedSlots] = {};

  // Runs launch(slot) with a slot acquired as above. The slot counts as used
  // whatever launch returns: it may fail behind a kernel that is queued
  // already and uses the slot's counters.
  template <typename F>
  typename Api::Status run(typename Api::Stream s, bool captured, F&& launch) {
    std::lock_guard<std::mutex> lock(mu);
    if (captured) return launch(sched_slot_of(graph_next++, true));
    const int slot = sched_slot_of(eager_next, false);
    typename Api::Event& ev = done[slot];
    const typename Api::Status ready = ev == typename Api::Event{} ? Api::create(&ev) : Api::wait(s, ev);
    if (ready != Api::kOk) return ready;
    const typename Api::Status r = launch(slot);
    ++eager_next;
    const typename Api::Status recorded = Api::record(ev, s);
    return r != Api::kOk ? r : recorded;
  }
};

}  // namespace sa
