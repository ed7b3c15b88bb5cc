"""Layers of hybrid linear-attention models on MI355X (gfx950) as hand-written HIP kernels behind a C ABI
(include/gdn.h, libgdn.so): the chunked gated delta rule, forward, deterministic
backward and the recurrent decode step, with its short convolution; linear attention
with a decay for each head; softmax attention with a sliding window and its paged
key-value cache; rotary positions; the root-mean-square norm. ``gdn`` is the
Python binding; importing it needs the built library (``python -m
chunked_gated_delta_04_amd.build``).
"""
