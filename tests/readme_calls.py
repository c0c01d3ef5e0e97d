"""The calls of README.md's C examples, with the parameter names that
include/q4k.h gives them."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _text(*path):
    with open(os.path.join(ROOT, *path)) as f:
        return re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)


def parameters():
    """Parameter names of every function that the header declares."""
    found = re.findall(r"\b(q[46]k_[a-z0-9_]+)\s*\(([^()]*)\)\s*;", _text("include", "q4k.h"))
    return {name: [re.search(r"(\w+)\s*$", p).group(1) for p in args.split(",")
                   if p.strip() not in ("", "void")] for name, args in found}


def blocks():
    """Per C example: its calls in order, as (function, {parameter: argument})."""
    names = parameters()
    out = []
    for code in re.findall(r"```c\n(.*?)```", _text("README.md"), flags=re.S):
        calls = []
        for name, args in re.findall(r"\b(q[46]k_[a-z0-9_]+)\(([^;]*)\);", code):
            args = [a.strip() for a in args.split(",")]
            assert len(args) == len(names[name]), (name, args)
            calls.append((name, dict(zip(names[name], args))))
        out.append(calls)
    return out
