"""Several host threads that call the library at the same time."""
from __future__ import annotations

import threading


def at_once(calls, repeats):
    """Each (function, arguments) of the library `repeats` times in a thread
    of its own: how many of its calls did not return QLORA_OK.  The functions
    leave the interpreter's lock, so with their arguments at hand they run
    beside one another."""
    refused, start = [0] * len(calls), threading.Barrier(len(calls))

    def run(i, fn, args):
        start.wait()
        for _ in range(repeats):
            if fn(*args) != 0:
                refused[i] += 1

    threads = [threading.Thread(target=run, args=(i, *c)) for i, c in enumerate(calls)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return refused
