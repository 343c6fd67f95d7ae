"""Imported for its effect: the library is there, built if nothing is."""
import os

from moe_experts_amd import build

if not os.path.exists(build.LIB):
    build.build()
