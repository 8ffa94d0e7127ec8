"""Functions run at once, a host thread each."""

from __future__ import annotations

import threading


def run_together(work, timeout=60.0):
    """Runs every function of ``work`` in a thread of its own, all let go together, and
    raises what the first of them raised, or TimeoutError where one has not come to its
    end in time. The threads are daemons: one that is stuck does not hold up the exit."""
    start, failed, done = threading.Barrier(len(work)), [], []

    def body(i, f):
        try:
            start.wait(timeout)
            f()
            done.append(i)
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=body, args=a, daemon=True) for a in enumerate(work)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout)
    if failed:
        raise failed[0]
    if len(done) < len(work) or any(t.is_alive() for t in threads):
        raise TimeoutError(f"{len(work) - len(done)} of {len(work)} threads have not ended")
