"""Runs one case of perf/more_operators.py three times through the library, for ncu.

    PYTHONPATH=. python profiles/bounded_context.py "window long train" len_lo=8192 len_hi=8192
"""
import importlib.util
import os
import sys

import torch


def main(name, *sizes):
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "perf", "more_operators.py")
    spec = importlib.util.spec_from_file_location("more_operators", path)
    cases = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(cases)
    cases.own = True
    case = next(dict(c) for c in cases.listed() if c["name"] == name)
    case.update((k, int(v)) for k, v in (x.split("=") for x in sizes))
    state = cases.prepare(case, 1)
    for _ in range(3):
        cases.run(state)
    torch.cuda.synchronize()


if __name__ == "__main__":
    main(*sys.argv[1:])
