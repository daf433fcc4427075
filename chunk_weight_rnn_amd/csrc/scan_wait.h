// When a tile of the recurrence (scan.hip) stops waiting for another one's word.
#pragma once

namespace e2ttt {

// Ticks of the 100 MHz wall clock and looks at the word.  A wait that lasts long means that the
// word will not come (another call was given the same workspace meanwhile) only if the wave
// was running: the clock goes on while a queue is set aside for another process's work, looks
// do not.  2^20 of them are a second or two at the 1 to 2 us that each takes.
constexpr unsigned long long kSpinTicks = 200000000;
constexpr unsigned kSpinLooks = 1u << 20;

constexpr bool gives_up(unsigned looks, unsigned long long ticks) { return looks >= kSpinLooks && ticks > kSpinTicks; }

}  // namespace e2ttt
