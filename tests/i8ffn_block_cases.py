"""Sizes at which the down projection for up to 16 tokens takes its row groups in several blocks.

(tokens, experts, slots, H, I, whether LDS holds the codes of all pairs)"""
CASES = [
    (16, 4, 16, 4112, 32, False),    # some workgroups have a second block, all of them several batches of pairs
    (16, 3, 16, 8208, 16, False),    # three blocks, the last of one row group; two batches
    (16, 3, 8, 8208, 16, True),      # two blocks of all pairs at once: the codes stay
    (6, 3, 8, 21520, 16, True),      # each workgroup quantises the hidden rows for itself
    (6, 3, 8, 21520, 512, True),     # the same, full units of codes
    (1, 4, 16, 65552, 32, True),     # one token
    (2, 4, 16, 65552, 16, True),
    (16, 3, 16, 4112, 1024, False),  # turns of four steps
    (16, 40, 16, 4112, 1024, False), # the same, many experts: chunks of fewer pairs
    (13, 5, 15, 6160, 48, False),    # odd counts of tokens and slots
    (16, 3, 16, 8208, 768, False),
    (1, 20, 16, 131072, 16, True),   # the longest row
]
