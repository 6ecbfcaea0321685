"""fp64 CPU oracle for exact attention — TEST INFRASTRUCTURE ONLY.

Only ``tests/``, ``__graft_entry__.smoke()`` and ``bench.py``'s cpu_baseline /
reference legs may import this package.  The CUDA library neither imports nor
links anything here; the two share no code.  See ``oracle/attention.py`` for
what each function computes, the passages it follows and how it is pinned, and
``oracle/paged.py`` for rotary positions and the paged cache.
"""
from .attention import *  # noqa: F401,F403
from .attention import __all__ as _attention
from .paged import *  # noqa: F401,F403
from .paged import __all__ as _paged

__all__ = _attention + _paged
