"""CPU oracle (test infrastructure only; see clover_oracle.py and moe_ops.py)."""
from .clover_oracle import *  # noqa: F401,F403
from . import moe_ops  # noqa: F401
